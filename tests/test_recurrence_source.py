"""What linear_recurrence.cu states about itself and no run can show, read from its source."""

import os
import re

import numpy as np

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


def horner(name):
    """The fp32 coefficients of the polynomial in `name`, highest power first, in 64 bits."""
    return [float(np.float32(c)) for c in re.findall(r"([-+]?\d\.\d{9}e[-+]\d\d)f", body(name))]


def test_the_polynomials_are_as_exact_as_their_comments_say():
    """log2(e) log1p(t) = t Q(t) on [0, 1], 2^y - 1 = y W(y) on [-1/2, 0]: the coefficients as rounded,
    evaluated in 64 bits (Horner of at most nine terms: 1e-15)"""
    t = np.linspace(0, 1, 20001)[1:]
    Q, W = horner("decay_gate"), horner("code_factor")
    assert len(Q) == 9 and len(W) == 5
    assert "(3.2e-8;" in SOURCE and "1.6e-8; fitted as above" in SOURCE
    assert np.abs(np.polyval(Q, t) * t / (np.log1p(t) / np.log(2.0)) - 1).max() <= 3.2e-8
    y = -0.5 * t
    assert np.abs(np.polyval(W, y) * y / np.expm1(y * np.log(2.0)) - 1).max() <= 1.6e-8
