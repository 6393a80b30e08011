"""fp64 CPU oracle of the trainable block around a recurrence: the gated linear recurrence with
its gradient, layer normalisation with its gradient, and the gradients of the short
convolution + SiLU and of the gated RMS normalisation.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle/``.

  linear_recurrence   h_t = exp(g_t) h_{t-1} + sigmoid(b_t) x_t per channel, with the rule's
                      decay g = -exp(A_log) softplus(a + dt_bias) (Mila "GatedDeltaRule.ixx
                      File Reference", Detailed Description), one token after the other
  *_backward          the chain rule written out; pinned by central differences in
                      ``tests/test_oracle_block.py``

Each gradient also comes as a magnitude (``*_magnitude``): the same sums over absolute
values, which is what rounding errors of the terms scale with where the terms cancel.
"""

from __future__ import annotations

import numpy as np

from .mixer_io import silu


def sigmoid(x):
    x = np.asarray(x, dtype=np.float64)
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, e) / (1.0 + e)


def softplus(x):
    x = np.asarray(x, dtype=np.float64)
    return np.maximum(x, 0.0) + np.log1p(np.exp(-np.abs(x)))


def silu_slope(x):
    s = sigmoid(x)
    return s * (1.0 + x * (1.0 - s))


def spans(B, T, cu_seqlens):
    """(batch row, first token, end token) of every sequence."""
    if cu_seqlens is None:
        return [(i, 0, T) for i in range(B)]
    return [(0, int(lo), int(hi)) for lo, hi in zip(cu_seqlens[:-1], cu_seqlens[1:])]


def linear_recurrence(x, a, b, A_log, dt_bias, init_state=None, cu_seqlens=None):
    """x, a, b [B, T, C]; returns (h [B, T, C], final state [Nseq, C]); rows outside the
    sequences are NaN."""
    x, a, b = (np.asarray(v, dtype=np.float64) for v in (x, a, b))
    g = -np.exp(np.asarray(A_log, np.float64)) * softplus(a + np.asarray(dt_bias, np.float64))
    lam, u = np.exp(g), sigmoid(b) * x
    sq = spans(*x.shape[:2], cu_seqlens)
    h = np.full(x.shape, np.nan)
    final = np.zeros((len(sq), x.shape[2]))
    if init_state is not None:
        final += np.asarray(init_state, np.float64)
    for n, (row, lo, hi) in enumerate(sq):
        for t in range(lo, hi):
            final[n] = lam[row, t] * final[n] + u[row, t]
            h[row, t] = final[n]
    return h, final


def linear_recurrence_backward(x, a, b, A_log, dt_bias, grad_out, grad_final=None,
                               init_state=None, cu_seqlens=None):
    """Gradients (dx, da, db, dA_log, ddt_bias, dinit) of
    sum(h * grad_out) + sum(final * grad_final)."""
    x, a, b = (np.asarray(v, dtype=np.float64) for v in (x, a, b))
    A, z = np.exp(np.asarray(A_log, np.float64)), a + np.asarray(dt_bias, np.float64)
    g = -A * softplus(z)
    lam, i = np.exp(g), sigmoid(b)
    h, _ = linear_recurrence(x, a, b, A_log, dt_bias, init_state, cu_seqlens)
    sq = spans(*x.shape[:2], cu_seqlens)
    init = (np.zeros((len(sq), x.shape[2])) if init_state is None
            else np.asarray(init_state, np.float64))
    dinit = (np.zeros_like(init) if grad_final is None
             else np.array(grad_final, dtype=np.float64))
    dx, da, db = (np.full(x.shape, np.nan) for _ in range(3))
    dA_log, ddt = np.zeros(x.shape[2]), np.zeros(x.shape[2])
    for n, (row, lo, hi) in enumerate(sq):
        for t in range(hi - 1, lo - 1, -1):
            D = dinit[n] + np.asarray(grad_out[row, t], np.float64)
            prev = h[row, t - 1] if t > lo else init[n]
            dx[row, t] = i[row, t] * D
            db[row, t] = D * x[row, t] * i[row, t] * sigmoid(-b[row, t])
            dg = D * prev * lam[row, t]
            da[row, t] = -A * sigmoid(z[row, t]) * dg
            dA_log += dg * g[row, t]
            ddt += da[row, t]
            dinit[n] = lam[row, t] * D
    return dx, da, db, dA_log, ddt, dinit


def recurrence_magnitude(x, a, b, A_log, dt_bias, grad_out, grad_final=None, init_state=None,
                         cu_seqlens=None):
    """|.|-versions of (h, final) and of the six gradients: every term of every sum counted
    with its absolute value."""
    mag = lambda v: None if v is None else np.abs(np.asarray(v, np.float64))  # noqa: E731
    h, final = linear_recurrence(mag(x), a, b, A_log, dt_bias, mag(init_state), cu_seqlens)
    grads = linear_recurrence_backward(mag(x), a, b, A_log, dt_bias, mag(grad_out),
                                       mag(grad_final), mag(init_state), cu_seqlens)
    return (h, final) + tuple(np.abs(v) for v in grads)


def layer_norm(x, weight, bias=None, eps=1e-5):
    """Rows of x [..., d]; returns (y, mean, rstd)."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    y = (x - mean[..., None]) * rstd[..., None] * np.asarray(weight, np.float64)
    return y if bias is None else y + np.asarray(bias, np.float64), mean, rstd


def layer_norm_backward(x, weight, grad_y, eps=1e-5):
    """(dx, dweight, dbias), weight's and bias's summed over all rows."""
    x, dy = np.asarray(x, np.float64), np.asarray(grad_y, np.float64)
    _, mean, rstd = layer_norm(x, weight, None, eps)
    xh = (x - mean[..., None]) * rstd[..., None]
    q = dy * np.asarray(weight, np.float64)
    dx = rstd[..., None] * (q - q.mean(-1, keepdims=True) -
                            xh * (q * xh).mean(-1, keepdims=True))
    axes = tuple(range(x.ndim - 1))
    return dx, (dy * xh).sum(axes), dy.sum(axes)


def short_conv_silu_backward(x, weight, grad_y, bias=None, state=None, grad_state_out=None):
    """(dx [B, T, C], dweight [C, W], dbias [C], dstate [B, C, W-1]) of the causal convolution
    + SiLU; grad_state_out is the gradient of the state after the call."""
    x, w, dy = (np.asarray(v, np.float64) for v in (x, weight, grad_y))
    B, T, C = x.shape
    W = w.shape[1]
    state = np.zeros((B, C, W - 1)) if state is None else np.asarray(state, np.float64)
    hist = np.concatenate([np.swapaxes(state, 1, 2), x], axis=1)
    s = np.zeros((B, T, C)) + (0.0 if bias is None else np.asarray(bias, np.float64))
    for i in range(W):
        s += w[:, i] * hist[:, i:i + T]
    ds = dy * silu_slope(s)
    dhist, dw = np.zeros_like(hist), np.zeros_like(w)
    for i in range(W):
        dhist[:, i:i + T] += w[:, i] * ds
        dw[:, i] = (ds * hist[:, i:i + T]).sum((0, 1))
    if grad_state_out is not None:
        dhist[:, T:] += np.swapaxes(np.asarray(grad_state_out, np.float64), 1, 2)
    return dhist[:, W - 1:], dw, ds.sum((0, 1)), np.swapaxes(dhist[:, :W - 1], 1, 2).copy()


def gated_rmsnorm_backward(o, z, weight, grad_y, eps=1e-6):
    """(do, dz, dweight) of o / sqrt(mean(o^2) + eps) * weight * SiLU(z)."""
    o, z, w, dy = (np.asarray(v, np.float64) for v in (o, z, weight, grad_y))
    r = 1.0 / np.sqrt((o * o).mean(-1, keepdims=True) + eps)
    q = dy * w * silu(z)
    do = r * q - o * r ** 3 * (q * o).mean(-1, keepdims=True)
    dz = dy * o * r * w * silu_slope(z)
    return do, dz, (dy * o * r * silu(z)).sum(tuple(range(o.ndim - 1)))
