"""The recurrent block as a model runs it: layer norm, projections, short convolution + SiLU,
gated linear recurrence, gated RMS norm per head.

Training: the block's gradients, chained through the backward calls, against torch's
autograd of the same block in 64 bits.  The calls hand bf16 tensors to one another (the normed
input, the projections, the convolution's output and every gradient of these), so a value
has passed up to eight roundings of at most 2^-8 on its way, of random sign: the relative
error of a whole gradient tensor stays below 8 x 2^-8, about 3 %.

Serving: a prompt and then single tokens, every state carried in place, against one pass
over all tokens."""

import numpy as np
import pytest

import gated_delta_rule_145_b200 as gdr

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
B, T, D, C, HEAD = 2, 150, 128, 192, 64


class Block:
    """Weights of one block and its two ways of running."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s, std=1.0: torch.randn(s, device="cuda", generator=g) * std  # noqa: E731
        self.w = dict(ln_w=1 + 0.1 * r(D), ln_b=0.1 * r(D), w_in=r(D, 3 * C, std=D ** -0.5),
                      w_z=r(D, C, std=D ** -0.5), conv_w=0.5 * r(3 * C, 4), conv_b=0.1 * r(3 * C),
                      A_log=torch.rand(C, device="cuda", generator=g) * 2,
                      dt_bias=r(C) - 2.0, norm_w=1 + 0.1 * r(HEAD))
        self.rand = r

    def forward(self, x, conv_state, state):
        """Library calls, bf16 between them; returns (y fp32 [B, T, C], what backward needs);
        conv_state and state are updated in place."""
        w, k = self.w, {}
        n, t = x.shape[0], x.shape[1]
        k["x"] = x
        k["n"], k["mean"], k["rstd"] = gdr.layer_norm(x, w["ln_w"], w["ln_b"])
        k["u"] = (k["n"].float() @ w["w_in"]).bfloat16()
        k["z"] = (k["n"].float() @ w["w_z"]).bfloat16()
        k["conv_state"], k["state"] = conv_state.clone(), state.clone()
        k["v"] = torch.empty_like(k["u"])
        gdr.gdr_short_conv_silu(k["u"], w["conv_w"], w["conv_b"], conv_state, conv_state, k["v"],
                                n, t, 3 * C)
        xs, a, b = k["v"].split(C, 2)
        k["h"], _ = gdr.linear_recurrence(xs, a, b, w["A_log"], w["dt_bias"], state,
                                          final_state=state)
        y = torch.empty_like(k["h"])
        gdr.gdr_gated_rmsnorm(k["h"], k["z"], w["norm_w"], y, n * t * C // HEAD, HEAD)
        return y, k

    def backward(self, k, dy):
        w, g = self.w, {}
        rows = lambda v: v.view(B, T, C // HEAD, HEAD)  # noqa: E731
        dh, dz, g["norm_w"] = gdr.gated_rmsnorm_backward(rows(k["h"]), rows(k["z"]), w["norm_w"],
                                                         rows(dy))
        dv = torch.empty_like(k["v"])
        (_, _, _, g["A_log"], g["dt_bias"], g["state"]) = gdr.linear_recurrence_backward(
            *k["v"].split(C, 2), w["A_log"], w["dt_bias"], k["h"], dh.view(B, T, C), None,
            k["state"], None, *dv.split(C, 2))
        du, g["conv_w"], g["conv_b"], g["conv_state"] = gdr.short_conv_silu_backward(
            k["u"], w["conv_w"], dv, w["conv_b"], k["conv_state"])
        dz = dz.view(B, T, C)
        n = k["n"].float().view(-1, D)
        g["w_in"] = n.t() @ du.float().view(-1, 3 * C)
        g["w_z"] = n.t() @ dz.float().view(-1, C)
        dn = (du.float() @ w["w_in"].t() + dz.float() @ w["w_z"].t()).bfloat16()
        g["x"], g["ln_w"], g["ln_b"] = gdr.layer_norm_backward(k["x"], w["ln_w"], k["mean"],
                                                              k["rstd"], dn)
        return g

    def reference(self, x, conv_state, state, dy):
        """(y, gradients) of the block in 64 bits by autograd."""
        leaf = {n: v.double().requires_grad_() for n, v in
                dict(self.w, x=x, conv_state=conv_state, state=state).items()}
        q = leaf["x"]
        q = (q - q.mean(-1, keepdim=True)) * (q.var(-1, unbiased=False, keepdim=True) + 1e-5).rsqrt()
        q = q * leaf["ln_w"] + leaf["ln_b"]
        u, z = q @ leaf["w_in"], q @ leaf["w_z"]
        hist = torch.cat([leaf["conv_state"].transpose(1, 2), u], 1)
        v = torch.nn.functional.silu(sum(hist[:, i:i + T] * leaf["conv_w"][:, i]
                                         for i in range(4)) + leaf["conv_b"])
        xs, a, b = v.split(C, 2)
        lam = torch.exp(-torch.exp(leaf["A_log"]) *
                        torch.nn.functional.softplus(a + leaf["dt_bias"]))
        h, hs = leaf["state"], []
        for t in range(T):
            h = lam[:, t] * h + torch.sigmoid(b[:, t]) * xs[:, t]
            hs.append(h)
        h = torch.stack(hs, 1).view(B, T, C // HEAD, HEAD)
        y = h * (h.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * leaf["norm_w"] * \
            torch.nn.functional.silu(z.view(B, T, C // HEAD, HEAD))
        y = y.view(B, T, C)
        names = list(leaf)
        return y, dict(zip(names, torch.autograd.grad(y, [leaf[n] for n in names], dy.double())))


def _off(a, b):
    return float((a.double() - b).norm() / b.norm())


def test_training_step_gradients():
    block = Block(1)
    x = block.rand(B, T, D).bfloat16()
    conv_state, state, dy = block.rand(B, 3 * C, 3), block.rand(B, C), block.rand(B, T, C)
    y, k = block.forward(x, conv_state.clone(), state.clone())
    grads = block.backward(k, dy)
    torch.cuda.synchronize()
    assert gdr.gdr_device_status() == gdr.GDR_OK
    ry, want = block.reference(x, conv_state, state, dy)
    limit = 8 * 2.0 ** -8
    assert _off(y, ry) <= limit
    assert set(want) == set(grads)
    for name, g in grads.items():
        assert _off(g.view(want[name].shape), want[name]) <= limit, name


def test_training_step_replayed_from_a_graph():
    """the whole step, forward and backward, captured and replayed: the direct run's bits"""
    block = Block(2)
    x = block.rand(B, T, D).bfloat16()
    conv_state, state, dy = block.rand(B, 3 * C, 3), block.rand(B, C), block.rand(B, T, C)

    def step():
        y, k = block.forward(x, conv_state.clone(), state.clone())
        return [y] + [v for _, v in sorted(block.backward(k, dy).items())]

    want = step()
    graph, cap = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cap):
        step()
    with torch.cuda.graph(graph, stream=cap):
        got = step()
    torch.cuda.current_stream().wait_stream(cap)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(want, got):
            assert torch.equal(p, q)
    del graph


@pytest.mark.parametrize("T0", [1, 100])
def test_prompt_then_single_tokens(T0):
    block = Block(3)
    x = block.rand(B, T, D).bfloat16()
    conv_state, state = torch.zeros(B, 3 * C, 3, device="cuda"), torch.zeros(B, C, device="cuda")
    whole, _ = block.forward(x, conv_state.clone(), state.clone())
    parts = [block.forward(x[:, :T0].contiguous(), conv_state, state)[0]]
    for t in range(T0, T0 + 12):
        parts.append(block.forward(x[:, t:t + 1].contiguous(), conv_state, state)[0])
    torch.cuda.synchronize()
    # the same bf16 values go through every call, except where a matrix product of another
    # shape rounds another way: one bf16 step of an input, 2^-8
    got = torch.cat(parts, 1)
    assert _off(got, whole[:, :T0 + 12].double()) <= 2.0 ** -8
