"""A call that fails leaves nothing behind for the next one."""

import pytest

import gated_delta_rule_145_b200 as gdr

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
A = 1 << 20  # a fake aligned address: the call below fails before any launch


def _out_of_memory():
    """a prefill whose workspace (2^22 blocks of 16 heads, 16 KB and more each) no device holds; its
    allocation is the first thing that the call does after its checks"""
    return gdr.gdr_prefill_chunked(A, A, A, A, A, A, A, None, A, None, None, 1, 1 << 28, 16, 16, 128,
                                   128, 32, check=False)


def test_an_error_is_reported_once():
    x, w = torch.randn(700, 1160, device="cuda"), torch.ones(1160, device="cuda")
    c = torch.randn(1, 40, 64, device="cuda")
    p = torch.zeros(64, device="cuda")
    want = gdr.layer_norm(x, w)[0], gdr.linear_recurrence(c, c, c, p, p)[0]
    for i, call in enumerate((lambda: gdr.layer_norm(x, w)[0],
                              lambda: gdr.linear_recurrence(c, c, c, p, p)[0])):
        assert _out_of_memory() == gdr.GDR_ERR_OOM
        assert torch.equal(call(), want[i])
    assert _out_of_memory() == gdr.GDR_ERR_OOM
    assert gdr.gdr_device_status() == gdr.GDR_OK
    z = torch.randn(90, 64, device="cuda")
    y = torch.empty_like(z)
    gdr.gdr_gated_rmsnorm_f32(z, z, w[:64].contiguous(), y, 90, 64)
    torch.cuda.synchronize()
