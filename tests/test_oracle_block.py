"""Pins of the fp64 oracle in oracle/block.py: gradients against central differences of the
forward functions, closed forms, and the step over a packed boundary."""

import numpy as np
import pytest

from oracle import block, mixer_io

RNG = np.random.default_rng(99)


def _numeric(f, v, step=1e-6):
    """Central differences of the scalar f at every element of v."""
    v = np.array(v, dtype=np.float64)
    g = np.zeros_like(v)
    for i in np.ndindex(v.shape):
        keep = v[i]
        v[i] = keep + step
        hi = f(v)
        v[i] = keep - step
        lo = f(v)
        v[i] = keep
        g[i] = (hi - lo) / (2 * step)
    return g


def _close(a, b):
    # central differences of O(1) functions at step 1e-6: truncation 1e-12, rounding 1e-10 / 1e-6
    assert np.allclose(a, b, rtol=0, atol=3e-8 * max(1.0, np.abs(b).max()) * 10)


@pytest.mark.parametrize("cu", [None, [0, 2, 2, 7]])
def test_recurrence_gradients_against_differences(cu):
    B, T, C = (2, 5, 3) if cu is None else (1, 7, 3)
    n = B if cu is None else len(cu) - 1
    x, a, b, go = (RNG.standard_normal((B, T, C)) for _ in range(4))
    A_log, dt = RNG.uniform(-1, 1, C), RNG.standard_normal(C)
    init, gf = RNG.standard_normal((n, C)), RNG.standard_normal((n, C))

    def loss(**kw):
        v = dict(x=x, a=a, b=b, A_log=A_log, dt_bias=dt, init_state=init)
        v.update(kw)
        h, f = block.linear_recurrence(**v, cu_seqlens=cu)
        return (h * go).sum() + (f * gf).sum()

    got = block.linear_recurrence_backward(x, a, b, A_log, dt, go, gf, init, cu)
    for name, g, v in zip(("x", "a", "b", "A_log", "dt_bias", "init_state"), got,
                          (x, a, b, A_log, dt, init)):
        _close(g, _numeric(lambda t, name=name: loss(**{name: t}), v))


def test_recurrence_without_decay_is_a_running_sum():
    x = RNG.standard_normal((1, 50, 4))
    big = np.full((1, 50, 4), 1e3)
    h, f = block.linear_recurrence(x, -big, big, np.zeros(4), np.zeros(4))
    assert np.allclose(h, np.cumsum(x, 1)) and np.allclose(f, x.sum(1))


def test_packed_sequences_are_separate_calls():
    x, a, b = (RNG.standard_normal((1, 9, 2)) for _ in range(3))
    A, dt, init = RNG.uniform(-1, 1, 2), RNG.standard_normal(2), RNG.standard_normal((3, 2))
    h, f = block.linear_recurrence(x, a, b, A, dt, init, [0, 4, 4, 9])
    for n, (lo, hi) in enumerate([(0, 4), (4, 4), (4, 9)]):
        hn, fn = block.linear_recurrence(x[:, lo:hi], a[:, lo:hi], b[:, lo:hi], A, dt,
                                         init[n:n + 1])
        assert np.array_equal(h[:, lo:hi], hn) and np.array_equal(f[n:n + 1], fn)


def test_layer_norm_gradients_against_differences():
    x, dy = RNG.standard_normal((3, 6)) + 2.0, RNG.standard_normal((3, 6))
    w, b = RNG.uniform(0.5, 1.5, 6), RNG.standard_normal(6)
    f = lambda x=x, w=w, b=b: (block.layer_norm(x, w, b)[0] * dy).sum()  # noqa: E731
    dx, dw, db = block.layer_norm_backward(x, w, dy)
    _close(dx, _numeric(lambda v: f(x=v), x))
    _close(dw, _numeric(lambda v: f(w=v), w))
    _close(db, _numeric(lambda v: f(b=v), b))


@pytest.mark.parametrize("T", [1, 2, 3, 6])
def test_conv_gradients_against_differences(T):
    B, C = 2, 3
    x, dy = RNG.standard_normal((B, T, C)), RNG.standard_normal((B, T, C))
    w, b = RNG.standard_normal((C, 4)), RNG.standard_normal(C)
    st, dst = RNG.standard_normal((B, C, 3)), RNG.standard_normal((B, C, 3))

    def f(x=x, w=w, b=b, st=st):
        y, s = mixer_io.short_conv_silu(x, w, b, st)
        return (y * dy).sum() + (s * dst).sum()

    dx, dw, db, ds = block.short_conv_silu_backward(x, w, dy, b, st, dst)
    _close(dx, _numeric(lambda v: f(x=v), x))
    _close(dw, _numeric(lambda v: f(w=v), w))
    _close(db, _numeric(lambda v: f(b=v), b))
    _close(ds, _numeric(lambda v: f(st=v), st))


def test_gated_rmsnorm_gradients_against_differences():
    o, z, dy = (RNG.standard_normal((3, 5)) for _ in range(3))
    w = RNG.uniform(0.5, 1.5, 5)
    f = lambda o=o, z=z, w=w: (mixer_io.gated_rmsnorm(o, z, w) * dy).sum()  # noqa: E731
    do, dz, dw = block.gated_rmsnorm_backward(o, z, w, dy)
    _close(do, _numeric(lambda v: f(o=v), o))
    _close(dz, _numeric(lambda v: f(z=v), z))
    _close(dw, _numeric(lambda v: f(w=v), w))


def test_a_planted_sign_is_seen():
    """the pin sees a wrong gradient: the decay's gradient with its sign turned"""
    x, a, b, go = (RNG.standard_normal((1, 4, 2)) for _ in range(4))
    A, dt = np.zeros(2), np.zeros(2)
    da = -block.linear_recurrence_backward(x, a, b, A, dt, go)[1]
    num = _numeric(lambda v: (block.linear_recurrence(x, v, b, A, dt)[0] * go).sum(), a)
    with pytest.raises(AssertionError):
        _close(da, num)
