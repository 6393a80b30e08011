"""The trainable block's calls past 2^31 elements: the last rows of tensors whose offsets do not fit
32 bits, against the oracle.  Tolerances as in the calls' own tests, rounded up: bf16 outputs
one step (2^-7) of the value, fp32 ones 1e-4 of the tensor's RMS."""

import numpy as np
import pytest

import gated_delta_rule_145_b200 as gdr
from oracle import block

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu, pytest.mark.slow]


def _fill(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(shape, device="cuda", dtype=dtype)
    flat = t.view(-1)
    for lo in range(0, flat.numel(), 1 << 28):
        part = flat[lo:lo + (1 << 28)]
        part.copy_(torch.randn(part.numel(), device="cuda", generator=g) * scale)
    return t


def _host(t):
    return t.float().cpu().numpy().astype(np.float64)


def _near(got, ref, bf16):
    got, rms = _host(got), np.sqrt(np.mean(ref * ref))
    tol = 1e-4 * rms + (2.0 ** -7 * np.abs(ref) if bf16 else 0.0)
    assert (np.abs(got - ref) <= tol).all(), np.max(np.abs(got - ref) / tol)


def test_recurrence_tail():
    C, tail = 8192, 700
    T = (1 << 31) // C + 40 + tail
    bf = torch.bfloat16
    x, a, b = (_fill((1, T, C), bf, s) for s in (1, 2, 3))
    go = _fill((1, T, C), torch.float32, 4)
    A, d, init, gf = _fill((C,), torch.float32, 5), _fill((C,), torch.float32, 6), \
        _fill((2, C), torch.float32, 7), _fill((2, C), torch.float32, 8)
    cu = torch.tensor([0, T - tail, T], device="cuda", dtype=torch.int32)
    out, final = gdr.linear_recurrence(x, a, b, A, d, init, cu)
    grads = gdr.linear_recurrence_backward(x, a, b, A, d, out, go, gf, init, cu)
    torch.cuda.synchronize()
    assert gdr.gdr_device_status() == gdr.GDR_OK
    ch = slice(0, C, 64)
    cut = [_host(t[:, T - tail:, ch]) for t in (x, a, b)]
    args = cut + [_host(A[ch]), _host(d[ch])]
    rh, rf = block.linear_recurrence(*args, _host(init[1:, ch]))
    rg = block.linear_recurrence_backward(*args, _host(go[:, T - tail:, ch]), _host(gf[1:, ch]),
                                          _host(init[1:, ch]))
    _near(out[:, T - tail:, ch], rh, False)
    _near(final[1:, ch], rf, False)
    for g, r in zip(grads[:3], rg[:3]):
        _near(g[:, T - tail:, ch], r, True)
    _near(grads[5][1:, ch], rg[5], False)


def test_layer_norm_tail():
    d = 6144
    rows = (1 << 31) // d + 300
    x, dy = _fill((rows, d), torch.bfloat16, 1), _fill((rows, d), torch.bfloat16, 2)
    w = 1 + _fill((d,), torch.float32, 3, 0.1)
    y, mean, rstd = gdr.layer_norm(x, w)
    dx, dw, db = gdr.layer_norm_backward(x, w, mean, rstd, dy)
    torch.cuda.synchronize()
    hx, hdy, hw = _host(x[-200:]), _host(dy[-200:]), _host(w)
    ry, _, _ = block.layer_norm(hx, hw)
    rdx, _, _ = block.layer_norm_backward(hx, hw, hdy)
    _near(y[-200:], ry, True)
    _near(dx[-200:], rdx, True)
    want = torch.zeros(d, device="cuda", dtype=torch.float64)
    for lo in range(0, rows, 1 << 14):
        want += dy[lo:lo + (1 << 14)].double().sum(0)
    _near(db, want.cpu().numpy(), False)


def test_conv_tail():
    C, B = 8192, 3
    T = (1 << 31) // (C * B) + 50
    x, dy = _fill((B, T, C), torch.bfloat16, 1), _fill((B, T, C), torch.bfloat16, 2)
    w = _fill((C, 4), torch.float32, 3, 0.5)
    dx = gdr.short_conv_silu_backward(x, w, dy)[0]
    torch.cuda.synchronize()
    ch, n = slice(0, C, 64), 300
    hx, hdy = _host(x[-1:, -n:, ch]), _host(dy[-1:, -n:, ch])
    ref = block.short_conv_silu_backward(hx, _host(w[ch]), hdy)[0]
    _near(dx[-1:, -n + 3:, ch], ref[:, 3:], True)


def test_gated_rmsnorm_tail():
    d = 128
    rows = (1 << 31) // d + 1000
    o, dy = _fill((rows, d), torch.float32, 1), _fill((rows, d), torch.float32, 2)
    z, w = _fill((rows, d), torch.bfloat16, 3), 1 + _fill((d,), torch.float32, 4, 0.1)
    do, dz, dw = gdr.gated_rmsnorm_backward(o, z, w, dy)
    torch.cuda.synchronize()
    ref = block.gated_rmsnorm_backward(_host(o[-500:]), _host(z[-500:]), _host(w), _host(dy[-500:]))
    _near(do[-500:], ref[0], False)
    _near(dz[-500:], ref[1], True)
