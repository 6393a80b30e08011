"""Layer normalisation and its gradient against the fp64 oracle, and the refusals.

Tolerances, from the arithmetic before any run: a row's sums have at most 32 roundings in a
chain (32 values per thread at most, then two trees of 5), 2^-19 of the sum of magnitudes; the
mean's error moves every xh, so xh's magnitude counts as X = (|x| + mean|x|) rstd.  Sums over
rows add a chain of one rounding per row.  A bf16 output adds half a step, 2^-8 of its value."""

import numpy as np
import pytest

import gated_delta_rule_145_b200 as gdr
from gated_delta_rule_145_b200 import synth
from oracle import block

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
E = 2.0 ** -19
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def make(rows, d, dtype, seed, offset=0.0, scale=1.0):
    rng = np.random.default_rng(seed)
    r = synth.round_to_bf16 if dtype == "bf16" else (lambda v: v)
    x = r((rng.standard_normal((rows, d)) * scale + offset).astype(np.float32))
    dy = r(rng.standard_normal((rows, d)).astype(np.float32))
    return x, dy, rng.uniform(0.5, 1.5, d).astype(np.float32), \
        rng.standard_normal(d).astype(np.float32)


def dev(v, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(v)).cuda().to(dtype)


def within(got, ref, tol, what):
    err = np.abs(got.float().cpu().numpy().astype(np.float64) - ref)
    assert (err <= tol).all(), f"{what}: worst {np.max(err / tol):.2f} x"


def check(x, dy, w, b, dtype, eps=1e-5):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    xd, dyd, wd = dev(x, dt), dev(dy, dt), dev(w)
    y, mean, rstd = gdr.layer_norm(xd, wd, None if b is None else dev(b), eps)
    dx, dw, db = gdr.layer_norm_backward(xd, wd, mean, rstd, dyd)
    torch.cuda.synchronize()
    ry, rm, rr = block.layer_norm(x, w, b, eps)
    rdx, rdw, rdb = block.layer_norm_backward(x, w, dy, eps)
    rows = x.shape[0]
    ax = np.abs(x.astype(np.float64))
    m1 = ax.mean(1, keepdims=True)
    X = (ax + m1) * rr[:, None]
    drift = 1 + X.max(1, keepdims=True) ** 2 * E  # rstd's own error, second order in the mean's
    half = HALF[dtype]
    within(mean, rm, E * m1[:, 0] + 1e-30, "mean")
    within(rstd, rr, 2 * E * drift[:, 0] * rr, "rstd")
    mag = X * np.abs(w) + (0 if b is None else np.abs(b))
    within(y, ry, 2 * E * drift * mag + half * np.abs(ry), "y")
    q = np.abs(dy * w).astype(np.float64)
    gmag = rr[:, None] * (q + q.mean(1, keepdims=True) + X * (q * X).mean(1, keepdims=True))
    within(dx, rdx, 4 * E * drift * gmag + half * np.abs(rdx), "dx")
    chain = E + rows * 2.0 ** -24
    within(dw, rdw, 2 * chain * (np.abs(dy) * X * drift).sum(0) + 1e-30, "dweight")
    within(db, rdb, chain * np.abs(dy.astype(np.float64)).sum(0) + 1e-30, "dbias")


# widths around one warp's narrow form (<= 256), around whole warps, one and several vectors
# per thread (8192, 16384 and above)
@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [
    (1, 8), (5, 16), (33, 24), (300, 64), (17, 136), (1000, 256), (3, 264), (64, 512),
    (700, 1024), (1001, 1160), (31, 4096), (200, 6144), (3, 8192), (5, 8200), (2, 16384),
    (3, 16392), (2, 32768), (601, 2056), (703, 4104), (1501, 6144), (640, 9216), (1201, 8200)])
def test_against_oracle(rows, d, dtype):
    check(*make(rows, d, dtype, rows * 31 + d), dtype)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_rows_than_a_grid(dtype):
    check(*make(20000, 40, dtype, 1), dtype)
    check(*make(5000, 264, dtype, 2), dtype)


@gpu
def test_without_bias_far_mean_constant_rows_and_large_values():
    x, dy, w, b = make(50, 520, "f32", 3, offset=300.0)
    check(x, dy, w, None, "f32")
    x, dy, w, b = make(50, 520, "f32", 4, scale=1e15)
    check(x, dy, w, b, "f32")
    x, dy, w, b = make(9, 136, "f32", 5)
    x[:] = 2.5  # no variance: rstd = 1 / sqrt(eps), xh = 0
    y, mean, rstd = gdr.layer_norm(dev(x), dev(w), dev(b), 1e-5)
    assert torch.equal(y, dev(b).expand(9, 136)) and (mean == 2.5).all()
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [(3, 3080), (700, 3600), (301, 4096), (5, 4104), (450, 6152), (77, 8192),
                                    (9, 8200)])
def test_columns_per_thread_edges(rows, d, dtype):
    """widths around those where a thread takes twice the columns, or an SM half the blocks"""
    check(*make(rows, d, dtype, rows + d), dtype)


@gpu
@pytest.mark.parametrize("d", [64, 1160, 6144, 20480])
def test_a_variance_whose_inverse_no_float_holds(d):
    """no eps and values of 1e-18: rstd times a gradient of 1e6 is a float, rstd^2 times it none"""
    x, dy, w, b = make(21, d, "f32", 8, scale=1e-18)
    check(x, dy * np.float32(1e6), w, b, "f32", 0.0)


@gpu
@pytest.mark.parametrize("d", [64, 1160, 20480])
def test_a_gradient_of_nan_stays_in_its_row(d):
    x, dy, w, b = make(40, d, "f32", 9)
    xd, wd = dev(x), dev(w)
    _, mean, rstd = gdr.layer_norm(xd, wd)
    clean = gdr.layer_norm_backward(xd, wd, mean, rstd, dev(dy))
    dy[6, 5] = np.nan
    dy[13, 2] = np.inf
    got = gdr.layer_norm_backward(xd, wd, mean, rstd, dev(dy))
    rows = [i for i in range(40) if i not in (6, 13)]
    cols = [i for i in range(d) if i not in (5, 2)]
    assert torch.equal(clean[0][rows], got[0][rows])
    assert torch.isnan(got[0][6]).all() and torch.isnan(got[1][5]) and torch.isnan(got[2][5])
    assert torch.equal(clean[1][cols], got[1][cols]) and torch.equal(clean[2][cols], got[2][cols])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 264, 1160, 4096, 6144, 8200, 20480])
def test_rows_of_one_value_add_nothing_to_the_weight_gradient(d, dtype):
    """x - mean is 0 exactly, so xh is, whatever rstd; grad_x = rstd (q - mean(q)) is left, to the
    tolerance of the test above without X (xh's magnitude)"""
    x, dy, w, _ = make(300, d, dtype, 10)
    x[:] = np.linspace(-3, 40, 300, dtype=np.float32)[:, None]
    x = synth.round_to_bf16(x)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    xd, wd = dev(x, dt), dev(w)
    _, mean, rstd = gdr.layer_norm(xd, wd)
    dx, dw, db = gdr.layer_norm_backward(xd, wd, mean, rstd, dev(dy, dt))
    torch.cuda.synchronize()
    assert torch.equal(mean, xd[:, 0].float()) and (dw == 0).all()
    q = dy.astype(np.float64) * w
    m = np.abs(q).mean(1, keepdims=True)
    ref = (q - q.mean(1, keepdims=True)) * 1e-5 ** -0.5
    within(dx, ref, 4 * E * (np.abs(q) + m) * 1e-5 ** -0.5 + HALF[dtype] * np.abs(ref), "dx")


@gpu
@pytest.mark.parametrize("d", [64, 1160])
def test_a_row_of_nan_stays_alone(d):
    x, dy, w, b = make(40, d, "f32", 6)
    clean = gdr.layer_norm(dev(x), dev(w), dev(b))
    x[7, 3] = np.nan
    x[9, 2] = np.inf
    got = gdr.layer_norm(dev(x), dev(w), dev(b))
    keep = [i for i in range(40) if i not in (7, 9)]
    for p, q in zip(clean, got):
        assert torch.equal(p[keep], q[keep])
    assert torch.isnan(got[0][7]).all() and torch.isnan(got[0][9]).any()


@gpu
@pytest.mark.parametrize("d,dtype", [(64, torch.float32), (1160, torch.bfloat16), (6144, torch.bfloat16)])
def test_in_place_again_and_from_a_graph(d, dtype):
    x, dy, w, b = make(700, d, "bf16", 7)
    xd, dyd, wd, bd = dev(x, dtype), dev(dy, dtype), dev(w), dev(b)
    y, mean, rstd = gdr.layer_norm(xd, wd, bd)
    want = gdr.layer_norm_backward(xd, wd, mean, rstd, dyd)
    same = xd.clone()
    assert gdr.layer_norm(same, wd, bd, y=same)[0] is same and torch.equal(same, y)
    g = dyd.clone()
    again = gdr.layer_norm_backward(xd, wd, mean, rstd, g, grad_x=g)
    for p, q in zip(want, again):
        assert torch.equal(p, q)
    graph, cap = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=cap):
        y2, m2, r2 = gdr.layer_norm(xd, wd, bd, stream=cap)
        g2 = gdr.layer_norm_backward(xd, wd, m2, r2, dyd, stream=cap)
    torch.cuda.current_stream().wait_stream(cap)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip((y, mean, rstd) + want, (y2, m2, r2) + g2):
            assert torch.equal(p, q)
    del graph


@gpu
def test_no_rows_and_skipped_outputs():
    w = torch.ones(64, device="cuda")
    e = torch.empty(0, 64, device="cuda")
    y, mean, rstd = gdr.layer_norm(e, w)
    dx, dw, db = gdr.layer_norm_backward(e, w, mean, rstd, e)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()
    x, dy, w, b = make(20, 264, "f32", 8)
    xd, wd, dyd = dev(x), dev(w), dev(dy)
    y, mean, rstd = gdr.layer_norm(xd, wd)
    y2, dx, dx2 = torch.empty_like(xd), torch.empty_like(xd), torch.empty_like(xd)
    dw = torch.empty(264, device="cuda")
    gdr.gdr_layer_norm_f32(xd, wd, None, y2, None, None, 20, 264)
    gdr.gdr_layer_norm_backward_f32(xd, wd, mean, rstd, dyd, dx, dw, None, 20, 264)
    gdr.gdr_layer_norm_backward_f32(xd, wd, mean, rstd, dyd, dx2, None, None, 20, 264)
    want = gdr.layer_norm_backward(xd, wd, mean, rstd, dyd)
    assert torch.equal(y, y2) and torch.equal(dx, want[0]) and torch.equal(dx2, want[0])
    assert torch.equal(dw, want[1])


A = 1 << 20  # fake aligned addresses: every call below fails a check before any launch


@pytest.mark.parametrize("suffix", ["", "_f32"])
def test_refusals(suffix):
    def fwd(**kw):
        args = dict(x=A, weight=A, bias=None, y=A, mean=None, rstd=None, rows=4, d=64, eps=1e-5)
        args.update(kw)
        return getattr(gdr, "gdr_layer_norm" + suffix)(**args, stream=0, check=False)

    def bwd(**kw):
        args = dict(x=A, weight=A, mean=A, rstd=A, grad_y=A, grad_x=A, grad_weight=A,
                    grad_bias=A, rows=4, d=64)
        args.update(kw)
        return getattr(gdr, "gdr_layer_norm_backward" + suffix)(**args, stream=0, check=False)

    for call, needed in ((fwd, "x weight y"), (bwd, "x weight mean rstd grad_y grad_x")):
        for p in needed.split():
            assert call(**{p: None}) == gdr.GDR_ERR_NULL, p
        for kw in (dict(rows=-1), dict(d=0), dict(d=4), dict(d=60)):
            assert call(**kw) == gdr.GDR_ERR_SHAPE, kw
        assert call(d=32776) == gdr.GDR_ERR_UNSUPPORTED
        for p in ("x", "weight"):
            assert call(**{p: A + 8}) == gdr.GDR_ERR_ALIGN, p
    # sizes that would wrap to others
    assert fwd(d=2 ** 32 + 64) == gdr.GDR_ERR_SHAPE == bwd(rows=2 ** 64 + 4)
    assert fwd(eps=-1.0) == gdr.GDR_ERR_SHAPE and fwd(eps=float("nan")) == gdr.GDR_ERR_SHAPE
    assert fwd(bias=A + 4) == gdr.GDR_ERR_ALIGN and fwd(y=A + 4) == gdr.GDR_ERR_ALIGN
    assert bwd(grad_y=A + 8) == gdr.GDR_ERR_ALIGN and bwd(grad_x=A + 8) == gdr.GDR_ERR_ALIGN


def test_binding_refuses_cpu_tensors():
    x, w = torch.zeros(4, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="CUDA"):
        gdr.layer_norm(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        gdr.layer_norm_backward(x, w, x[:, 0], x[:, 0], x)
