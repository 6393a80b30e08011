"""Every output of the trainable block's calls between two guard ranges of a marker value that must
survive, with the inputs unchanged: a stray write of a tile's ragged edge would show."""

import numpy as np
import pytest

import gated_delta_rule_145_b200 as gdr

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
GUARD, MARK = 4096, 12345.0


class Guarded:
    """Buffers of the wanted shape inside larger ones filled with the marker."""

    def __init__(self):
        self.all = []

    def __call__(self, *shape, dtype=torch.float32):
        n = int(np.prod(shape))
        n16 = (n + 15) // 16 * 16
        buf = torch.full((GUARD + n16 + GUARD,), MARK, device="cuda", dtype=dtype)
        self.all.append((buf, n))
        return buf[GUARD:GUARD + n].view(shape)

    def check(self):
        torch.cuda.synchronize()
        for buf, n in self.all:
            mark = torch.full((), MARK, dtype=buf.dtype).item()
            assert (buf[:GUARD] == mark).all() and (buf[GUARD + n:] == mark).all()
            assert torch.isfinite(buf[GUARD:GUARD + n].float()).all()
            assert not (buf[GUARD:GUARD + n] == mark).all() or n == 0


def _inputs(*specs):
    g = torch.Generator(device="cuda").manual_seed(11)
    return [torch.randn(s, device="cuda", generator=g).to(d) for s, d in specs]


F, H = torch.float32, torch.bfloat16


@pytest.mark.parametrize("dtype", [H, F])
@pytest.mark.parametrize("B,T,C", [(1, 1, 8), (3, 50, 72), (2, 200, 136), (1, 3001, 8), (2, 777, 1160),
                                   (1, 5000, 6152)])
def test_recurrence(B, T, C, dtype):
    x, a, b, go = _inputs(((B, T, C), dtype), ((B, T, C), dtype), ((B, T, C), dtype), ((B, T, C), F))
    A, d, init, gf = _inputs(((C,), F), ((C,), F), ((B, C), F), ((B, C), F))
    ins = [x, a, b, go, A, d, init, gf]
    kept = [v.clone() for v in ins]
    g = Guarded()
    out, final = g(B, T, C), g(B, C)
    grads = [g(B, T, C, dtype=dtype) for _ in range(3)]
    gA, gd, gi = g(C), g(C), g(B, C)
    f32 = dtype == F
    (gdr.gdr_linear_recurrence_f32 if f32 else gdr.gdr_linear_recurrence)(
        x, a, b, A, d, init, out, final, None, B, T, C, C)
    (gdr.gdr_linear_recurrence_backward_f32 if f32 else gdr.gdr_linear_recurrence_backward)(
        x, a, b, A, d, init, out, go, gf, *grads, gA, gd, gi, None, B, T, C, C, C)
    g.check()
    for v, w in zip(ins, kept):
        assert torch.equal(v, w)
    assert gdr.gdr_device_status() == gdr.GDR_OK


@pytest.mark.parametrize("dtype", [H, F])
@pytest.mark.parametrize("rows,d", [(1, 8), (77, 136), (700, 264), (650, 1160), (5, 6144),
                                    (601, 8200), (3, 20000)])
def test_layer_norm(rows, d, dtype):
    x, dy, w, b = _inputs(((rows, d), dtype), ((rows, d), dtype), ((d,), F), ((d,), F))
    kept = [v.clone() for v in (x, dy, w, b)]
    g = Guarded()
    y, mean, rstd = g(rows, d, dtype=dtype), g(rows), g(rows)
    dx, dw, db = g(rows, d, dtype=dtype), g(d), g(d)
    f32 = dtype == F
    (gdr.gdr_layer_norm_f32 if f32 else gdr.gdr_layer_norm)(x, w, b, y, mean, rstd, rows, d)
    (gdr.gdr_layer_norm_backward_f32 if f32 else gdr.gdr_layer_norm_backward)(
        x, w, mean, rstd, dy, dx, dw, db, rows, d)
    g.check()
    for v, k in zip((x, dy, w, b), kept):
        assert torch.equal(v, k)


@pytest.mark.parametrize("B,T,C", [(1, 1, 8), (2, 5, 72), (3, 300, 136), (1, 2000, 1160)])
def test_conv(B, T, C):
    x, dy = _inputs(((B, T, C), H), ((B, T, C), H))
    w, b, st, ds = _inputs(((C, 4), F), ((C,), F), ((B, C, 3), F), ((B, C, 3), F))
    kept = [v.clone() for v in (x, dy, w, b, st, ds)]
    g = Guarded()
    dx, dw, db, dst = g(B, T, C, dtype=H), g(C, 4), g(C), g(B, C, 3)
    gdr.gdr_short_conv_silu_backward(x, w, b, st, dy, ds, dx, dw, db, dst, B, T, C)
    g.check()
    for v, k in zip((x, dy, w, b, st, ds), kept):
        assert torch.equal(v, k)


@pytest.mark.parametrize("rows,d,dtype", [(1, 32, H), (777, 64, F), (5000, 128, H)])
def test_gated_rmsnorm(rows, d, dtype):
    o, dy, z, w = _inputs(((rows, d), F), ((rows, d), F), ((rows, d), dtype), ((d,), F))
    kept = [v.clone() for v in (o, dy, z, w)]
    g = Guarded()
    do, dz, dw = g(rows, d), g(rows, d, dtype=dtype), g(d)
    (gdr.gdr_gated_rmsnorm_backward_f32 if dtype == F else gdr.gdr_gated_rmsnorm_backward)(
        o, z, w, dy, do, dz, dw, rows, d)
    g.check()
    for v, k in zip((o, dy, z, w), kept):
        assert torch.equal(v, k)
