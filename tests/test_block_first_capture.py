"""A process whose first call of every kind is made inside a stream capture: the library sets up its
pool, its attributes and its occupancy queries there without invalidating the capture."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import torch
import gated_delta_rule_145_b200 as gdr
bf = torch.bfloat16
r = lambda *s: torch.randn(s, device="cuda")
x, a, b, go, A = r(1, 5000, 6144).to(bf), r(1, 5000, 6144).to(bf), r(1, 5000, 6144).to(bf), \\
    r(1, 5000, 6144), r(6144)
u, w, n, o, l = r(3, 300, 136).to(bf), r(136, 4), r(136), r(500, 64), r(64)
q, ab, H = r(1, 300, 2, 128).to(bf), r(1, 300, 2).to(bf), r(2)

def run():
    out, final = gdr.linear_recurrence(x, a, b, A, A)
    got = [out, final, *gdr.linear_recurrence_backward(x, a, b, A, A, out, go)]
    got += gdr.short_conv_silu_backward(u, w, u)
    y, mean, rstd = gdr.layer_norm(u, n)
    got += [y, *gdr.layer_norm_backward(u, n, mean, rstd, u)]
    got += gdr.gated_rmsnorm_backward(o, o, l, o)
    return got + list(gdr.prefill(q, q, q, ab, ab, H, H))

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
assert gdr.gdr_device_status() == gdr.GDR_OK
for p, v in zip(got, run()):
    assert torch.equal(p, v)
print("same")
"""


def test_first_calls_inside_a_capture():
    p = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert p.returncode == 0 and "same" in p.stdout, p.stderr[-2000:]
