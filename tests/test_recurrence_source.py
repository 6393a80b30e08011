"""What linear_recurrence.cu states about itself and no run can show, read from its source."""

import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
with open(os.path.join(ROOT, "gated_delta_rule_145_b200", "csrc", "linear_recurrence.cu")) as f:
    SOURCE = f.read()


def body(name):
    """The text of the function `name`, from its opening brace to the closing one."""
    at = SOURCE.index("{", re.search(r"\b%s\([^;{]*\)\s*{" % name, SOURCE).start())
    depth, end = 0, at
    while depth or end == at:
        depth += {"{": 1, "}": -1}.get(SOURCE[end], 0)
        end += 1
    return SOURCE[at:end]


def test_what_peers_stored_is_waited_for_at_cluster_scope():
    """st.async from another CTA of the cluster releases at cluster scope; only an acquire that
    covers the writer orders its data before the reads behind the wait"""
    waits = re.findall(r"(\w+)\(&sm\.peers_in\[", SOURCE)
    assert [w for w in waits if w not in ("mbar_init", "peers_wait")] == [] and "peers_wait" in waits
    for name in ("peers_wait", "peers_wait_slow"):
        assert "peers_test(" in body(name) and "mbar_" not in body(name)
    assert "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64" in body("peers_test")
