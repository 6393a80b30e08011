"""Gradients of the short convolution + SiLU and of the gated RMS normalisation against the
fp64 oracle, and their refusals.

Tolerances, from the arithmetic before any run.  sigmoid from the special-function unit is off
by ~2^-20, so ds = dy f(s) by E = |dy| 2^-18 (1 + M), M = |bias| + sum |w x| (what s's roundings
scale with; |f'| and |f| stay below 1.2); sums of four or of many terms keep that factor, doubled for
the roundings of a sum's chain.  A bf16 output adds half a step, 2^-8 of its value."""

import numpy as np
import pytest

import gated_delta_rule_145_b200 as gdr
from gated_delta_rule_145_b200 import synth
from oracle import block, mixer_io

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
H = 2.0 ** -8


def dev(v, dtype=torch.float32):
    return None if v is None else torch.from_numpy(np.ascontiguousarray(v)).cuda().to(dtype)


def within(got, ref, tol, what):
    err = np.abs(got.float().cpu().numpy().astype(np.float64) - ref)
    assert (err <= tol).all(), f"{what}: worst {np.max(err / tol):.2f} x"


def conv_case(B, T, C, bias, state, seed=0):
    rng = np.random.default_rng(seed + T * 13 + C)
    f = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    return dict(x=synth.round_to_bf16(f(B, T, C)), w=f(C, 4) * 0.5,
                dy=synth.round_to_bf16(f(B, T, C)), bias=f(C) if bias else None,
                state=f(B, C, 3) if state else None, ds=f(B, C, 3) if state else None)


def conv_gpu(m):
    return gdr.short_conv_silu_backward(dev(m["x"], torch.bfloat16), dev(m["w"]),
                                        dev(m["dy"], torch.bfloat16), dev(m["bias"]),
                                        dev(m["state"]), dev(m["ds"]))


def conv_check(m, got):
    x, w, dy = (m[k].astype(np.float64) for k in ("x", "w", "dy"))
    B, T, C = x.shape
    ref = block.short_conv_silu_backward(x, w, dy, m["bias"], m["state"], m["ds"])
    st = np.zeros((B, C, 3)) if m["state"] is None else m["state"].astype(np.float64)
    hist = np.abs(np.concatenate([np.swapaxes(st, 1, 2), x], 1))
    M = sum(np.abs(w[:, i]) * hist[:, i:i + T] for i in range(4))
    M = M + (0 if m["bias"] is None else np.abs(m["bias"]))
    E = np.abs(dy) * 2.0 ** -18 * (1 + M)
    full = 1.2 * np.abs(dy) + E  # |ds|
    dh = np.zeros_like(hist)
    for i in range(4):
        dh[:, i:i + T] += np.abs(w[:, i]) * (2 * E + 2.0 ** -22 * full)
    if m["ds"] is not None:
        dh[:, T:] += 2.0 ** -22 * np.abs(np.swapaxes(m["ds"], 1, 2))
    chain = 2.0 ** -19
    dw = np.stack([((2 * E + chain * full) * hist[:, i:i + T]).sum((0, 1)) for i in range(4)], 1)
    within(got[0], ref[0], dh[:, 3:] + H * np.abs(ref[0]) + 1e-30, "dx")
    within(got[1], ref[1], dw + 1e-30, "dweight")
    within(got[2], ref[2], (2 * E + chain * full).sum((0, 1)) + 1e-30, "dbias")
    within(got[3], ref[3], np.swapaxes(dh[:, :3], 1, 2) + 1e-30, "dstate")


# lengths below the taps, around a warp's segment and a CTA's rows; channel tails of 8
CONV = [(1, 1, 8), (2, 2, 16), (3, 3, 64), (2, 4, 128), (1, 61, 136), (2, 64, 96), (1, 65, 1160),
        (2, 67, 8), (3, 200, 64), (1, 511, 128), (2, 777, 1160), (1, 2100, 72), (70, 5, 64),
        (20001, 3, 8)]  # more segments than a grid takes at once


@gpu
@pytest.mark.parametrize("bias,state", [(True, True), (False, False), (False, True)])
@pytest.mark.parametrize("B,T,C", CONV)
def test_conv(B, T, C, bias, state):
    m = conv_case(B, T, C, bias, state)
    got = conv_gpu(m)
    torch.cuda.synchronize()
    conv_check(m, got)


@gpu
@pytest.mark.parametrize("T0", [2, 100, 512])
def test_conv_chained_through_the_state_is_one_call(T0):
    """the second part's state gradient, handed to the first part's call, gives the
    gradients of one call over both parts"""
    m = conv_case(2, T0 + 40, 72, True, True, seed=9)
    cut = dict(m, x=m["x"][:, T0:], dy=m["dy"][:, T0:])
    _, mid = mixer_io.short_conv_silu(m["x"][:, :T0], m["w"], m["bias"], m["state"])
    cut["state"] = mid.astype(np.float32)
    second = conv_gpu(cut)
    first = conv_gpu(dict(m, x=m["x"][:, :T0], dy=m["dy"][:, :T0],
                          ds=second[3].cpu().numpy()))
    torch.cuda.synchronize()
    ref = block.short_conv_silu_backward(m["x"], m["w"], m["dy"], m["bias"], m["state"], m["ds"])
    scale = np.abs(ref[1]).max()
    assert np.abs((first[1] + second[1]).cpu().numpy() - ref[1]).max() <= 1e-4 * scale
    got = torch.cat([first[0], second[0]], 1).float().cpu().numpy()
    assert (np.abs(got - ref[0]) <= H * np.abs(ref[0]) + 1e-4).all()
    assert np.abs(first[3].cpu().numpy() - ref[3]).max() <= 1e-4


@gpu
@pytest.mark.parametrize("T", [9, 300])
def test_conv_nan_and_infinity_stay_in_their_channels(T):
    """a lane holds four channels: a NaN or an infinite sum of one is not another's"""
    m = conv_case(2, T, 72, True, True, seed=4)
    m["x"][0, 4, 3] = np.nan
    m["x"][1, 5, 8] = np.inf
    m["dy"][0, 6, 20] = np.nan
    m["bias"][31] = -np.inf
    m["bias"][40] = np.nan
    got = conv_gpu(m)
    torch.cuda.synchronize()
    keep = np.array([c for c in range(72) if c not in (3, 8, 20, 31, 40)])
    at = torch.from_numpy(keep).cuda()
    axis = dict(x=2, w=0, dy=2, bias=0, state=1, ds=1)
    conv_check({k: v.take(keep, axis[k]) for k, v in m.items()},
               [v.index_select(d, at) for v, d in zip(got, (2, 0, 0, 1))])
    assert torch.isnan(got[0][0, 4, 3]) and torch.isnan(got[2][[3, 20, 40]]).all()


@gpu
def test_conv_of_no_tokens_and_skipped_outputs():
    e = torch.empty(2, 0, 16, device="cuda", dtype=torch.bfloat16)
    w, ds = torch.ones(16, 4, device="cuda"), torch.randn(2, 16, 3, device="cuda")
    dx, dw, db, dst = gdr.short_conv_silu_backward(e, w, e, None, None, ds)
    assert torch.equal(dst, ds) and (dw == 0).all() and (db == 0).all()
    assert (gdr.short_conv_silu_backward(e, w, e)[3] == 0).all()
    m = conv_case(2, 70, 72, True, True)
    want = conv_gpu(m)
    dx = torch.empty_like(want[0])
    gdr.gdr_short_conv_silu_backward(dev(m["x"], torch.bfloat16), dev(m["w"]), dev(m["bias"]),
                                     dev(m["state"]), dev(m["dy"], torch.bfloat16), dev(m["ds"]),
                                     dx, None, None, None, 2, 70, 72)
    torch.cuda.synchronize()
    assert torch.equal(dx, want[0])


@gpu
@pytest.mark.parametrize("B,T,C", [(3, 300, 136), (1, 1, 64)])
def test_conv_again_and_from_a_graph(B, T, C):
    m = conv_case(B, T, C, True, True)
    want = conv_gpu(m)
    args = (dev(m["x"], torch.bfloat16), dev(m["w"]), dev(m["dy"], torch.bfloat16),
            dev(m["bias"]), dev(m["state"]), dev(m["ds"]))
    graph, cap = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=cap):
        got = gdr.short_conv_silu_backward(*args, stream=cap)
    torch.cuda.current_stream().wait_stream(cap)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(want, got):
            assert torch.equal(p, q)
    del graph


@gpu
@pytest.mark.parametrize("rows,d,zf32", [(1, 32, False), (7, 64, True), (33, 128, False),
                                         (3001, 64, True), (3001, 32, False),
                                         (20000, 128, False), (5, 128, True)])
def test_gated_rmsnorm(rows, d, zf32):
    rng = np.random.default_rng(rows + d)
    o, z, dy = (rng.standard_normal((rows, d)).astype(np.float32) for _ in range(3))
    z *= 3
    if not zf32:
        z = synth.round_to_bf16(z)
    w = rng.uniform(0.5, 1.5, d).astype(np.float32)
    o[0] = 0  # a row of zeros: r = 1 / sqrt(eps)
    got = gdr.gated_rmsnorm_backward(dev(o), dev(z, torch.float32 if zf32 else torch.bfloat16),
                                     dev(w), dev(dy))
    torch.cuda.synchronize()
    do, dz, dw = block.gated_rmsnorm_backward(o, z, w, dy)
    o, z, dy = (v.astype(np.float64) for v in (o, z, dy))
    r = 1 / np.sqrt((o * o).mean(1, keepdims=True) + 1e-6)
    q = np.abs(dy * w * mixer_io.silu(z))
    E = 2.0 ** -18
    within(got[0], do, E * (r * q + np.abs(o) * r ** 3 * (q * np.abs(o)).mean(1, keepdims=True)) +
           1e-30, "do")
    within(got[1], dz, E * np.abs(dy * o * r * w) * (1 + np.abs(z)) +
           (2.0 ** -24 if zf32 else H) * np.abs(dz) + 1e-30, "dz")
    terms = np.abs(dy * o * r * mixer_io.silu(z)).sum(0)
    within(got[2], dw, (E + rows / 64 * 2.0 ** -24) * 2 * terms + 1e-30, "dweight")


@gpu
@pytest.mark.parametrize("zf32", [False, True])
@pytest.mark.parametrize("scale,eps", [(1e12, 1e-6), (1e15, 1e-6), (1e17, 1e-6), (1e-13, 0.0),
                                       (1e-17, 0.0)])
def test_gated_rmsnorm_of_rows_whose_cubed_norm_no_float_holds(scale, eps, zf32):
    """r^3 underflows for large rows and overflows for small ones, the gradient does not; the
    tolerance is that of the test above with n = o r in the place of o (every factor that is
    rounded is of the size of a factor there)"""
    rng = np.random.default_rng(6)
    rows, d = 90, 64
    n, z, q = (rng.standard_normal((rows, d)).astype(np.float32) for _ in range(3))
    o = n * np.float32(scale)
    if not zf32:
        z = synth.round_to_bf16(z)
    dy = q + n * np.sign(z)  # a part along o, so that the second term counts
    w = rng.uniform(0.5, 1.5, d).astype(np.float32)
    got = gdr.gated_rmsnorm_backward(dev(o), dev(z, torch.float32 if zf32 else torch.bfloat16),
                                     dev(w), dev(dy), eps)
    torch.cuda.synchronize()
    do, dz, dw = block.gated_rmsnorm_backward(o, z, w, dy, eps)
    o, z, dy = (v.astype(np.float64) for v in (o, z, dy))
    r = 1 / np.sqrt((o * o).mean(1, keepdims=True) + eps)
    n, q = o * r, np.abs(dy * w * mixer_io.silu(z))
    E = 2.0 ** -18
    within(got[0], do, E * r * (q + np.abs(n) * (q * np.abs(n)).mean(1, keepdims=True)), "do")
    within(got[1], dz, E * np.abs(dy * n * w) * (1 + np.abs(z)) +
           (2.0 ** -24 if zf32 else H) * np.abs(dz) + 1e-30, "dz")
    terms = np.abs(dy * n * mixer_io.silu(z)).sum(0)
    within(got[2], dw, (E + rows / 64 * 2.0 ** -24) * 2 * terms + 1e-30, "dweight")


@gpu
@pytest.mark.parametrize("zf32", [False, True])
@pytest.mark.parametrize("lo,hi", [(-80, -20), (-20, -4), (-4, 4), (4, 90)])
def test_gated_rmsnorm_keeps_the_gate_to_fp32_rounding(lo, hi, zf32):
    """one row of ones without eps: r = 1 and n = 1 exactly, so dweight is SiLU(z) as computed:
    an exponential of at most two ulps (2^-22), a sum, a quotient and a product (2^-24 each):
    below 2^-21 of each value"""
    ones = torch.ones(1, 128, device="cuda")
    for seed in range(4):
        z = np.random.default_rng(seed).uniform(lo, hi, (1, 128)).astype(np.float32)
        if not zf32:
            z = synth.round_to_bf16(z)
        zd = dev(z, torch.float32 if zf32 else torch.bfloat16)
        dw = gdr.gated_rmsnorm_backward(ones, zd, ones[0], ones, 0.0)[2]
        ref = mixer_io.silu(z[0].astype(np.float64))
        within(dw, ref, 2.0 ** -21 * np.abs(ref) + 1e-36, "dweight")


@gpu
def test_gated_rmsnorm_in_place_and_no_rows():
    rng = np.random.default_rng(3)
    o, z, dy = (dev(rng.standard_normal((100, 64)).astype(np.float32)) for _ in range(3))
    w = torch.ones(64, device="cuda")
    want = gdr.gated_rmsnorm_backward(o, z, w, dy)
    g, gz, dw = dy.clone(), z.clone(), torch.empty(64, device="cuda")
    gdr.gdr_gated_rmsnorm_backward_f32(o, gz, w, g, g, gz, dw, 100, 64)
    torch.cuda.synchronize()
    assert torch.equal(g, want[0]) and torch.equal(gz, want[1]) and torch.equal(dw, want[2])
    e = torch.empty(0, 64, device="cuda")
    assert (gdr.gated_rmsnorm_backward(e, e, w, e)[2] == 0).all()


A = 1 << 20  # fake aligned addresses: every call below fails a check before any launch


def test_conv_refusals():
    def call(**kw):
        args = dict(x=A, weight=A, bias=None, conv_state_in=None, grad_y=A,
                    grad_conv_state_out=None, grad_x=A, grad_weight=A, grad_bias=A,
                    grad_conv_state_in=None, B=1, T=16, C=64, width=4)
        args.update(kw)
        return gdr.gdr_short_conv_silu_backward(**args, stream=0, check=False)

    for p in ("x", "weight", "grad_y", "grad_x"):
        assert call(**{p: None}) == gdr.GDR_ERR_NULL, p
    for kw in (dict(B=0), dict(T=-1), dict(C=0), dict(C=60), dict(B=1 << 24, T=64),
               dict(T=2 ** 31 - 1, C=8)):
        assert call(**kw) == gdr.GDR_ERR_SHAPE, kw
    assert call(width=3) == gdr.GDR_ERR_UNSUPPORTED
    for p in ("x", "grad_y", "grad_x", "weight"):
        assert call(**{p: A + 8}) == gdr.GDR_ERR_ALIGN, p
    for p in ("bias", "conv_state_in", "grad_conv_state_out", "grad_weight", "grad_bias",
              "grad_conv_state_in"):
        assert call(**{p: A + 2}) == gdr.GDR_ERR_ALIGN, p


@pytest.mark.parametrize("suffix", ["", "_f32"])
def test_gated_rmsnorm_refusals(suffix):
    def call(**kw):
        args = dict(o=A, z=A, weight=A, grad_y=A, grad_o=A, grad_z=A, grad_weight=A, rows=4, d=64,
                    eps=1e-6)
        args.update(kw)
        return getattr(gdr, "gdr_gated_rmsnorm_backward" + suffix)(**args, stream=0, check=False)

    for p in ("o", "z", "weight", "grad_y", "grad_o", "grad_z", "grad_weight"):
        assert call(**{p: None}) == gdr.GDR_ERR_NULL, p
    assert call(rows=-1) == gdr.GDR_ERR_SHAPE and call(eps=-1.0) == gdr.GDR_ERR_SHAPE
    assert call(d=96) == gdr.GDR_ERR_UNSUPPORTED
    for p in ("o", "grad_y", "grad_o", "weight"):
        assert call(**{p: A + 8}) == gdr.GDR_ERR_ALIGN, p
    assert call(z=A + 4) == gdr.GDR_ERR_ALIGN and call(grad_z=A + 4) == gdr.GDR_ERR_ALIGN


def test_binding_refuses_cpu_tensors():
    x, w = torch.zeros(1, 4, 8, dtype=torch.bfloat16), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="CUDA"):
        gdr.short_conv_silu_backward(x, w, x)
    o = torch.zeros(4, 32)
    with pytest.raises(ValueError, match="CUDA"):
        gdr.gated_rmsnorm_backward(o, o, o[0], o)
