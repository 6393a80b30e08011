"""The trainable block's calls beside autograd: they are not recorded, so a tensor whose gradient would be
lost is refused; from an autograd function they give the gradients."""

import pytest

import gated_delta_rule_145_b200 as gdr

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _calls():
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    x, p, w, c = r(2, 5, 64), r(64), r(64, 4), r(2, 5, 64).bfloat16()
    m = r(2, 5)
    return {
        "linear_recurrence": (gdr.linear_recurrence, [x, x.clone(), x.clone(), p, p.clone(), r(2, 64)]),
        "linear_recurrence_backward": (gdr.linear_recurrence_backward,
                                       [x, x.clone(), x.clone(), p, p.clone(), x.clone(), x.clone()]),
        "layer_norm": (gdr.layer_norm, [x, p, p.clone()]),
        "layer_norm_backward": (gdr.layer_norm_backward, [x, p, m, m.clone(), x.clone()]),
        "short_conv_silu_backward": (gdr.short_conv_silu_backward, [c, w, c.clone(), p]),
        "gated_rmsnorm_backward": (gdr.gated_rmsnorm_backward, [x, x.clone(), p, x.clone()]),
    }


@pytest.mark.parametrize("name", ["linear_recurrence", "linear_recurrence_backward", "layer_norm",
                                  "layer_norm_backward", "short_conv_silu_backward",
                                  "gated_rmsnorm_backward"])
def test_a_gradient_that_would_be_lost_is_refused(name):
    fn, args = _calls()[name]
    for i in range(len(args)):
        mine = [t.clone() for t in args]
        mine[i].requires_grad_()
        with pytest.raises(ValueError, match="autograd"):
            fn(*mine)
        with torch.no_grad():
            kept = fn(*mine)
        for p, q in zip(kept, fn(*args)):
            assert torch.equal(p, q) and not p.requires_grad


def test_gradients_through_an_autograd_function():
    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, b):
            y, mean, rstd = gdr.layer_norm(x, w, b)
            ctx.save_for_backward(x, w, mean, rstd)
            return y

        @staticmethod
        def backward(ctx, dy):
            return gdr.layer_norm_backward(*ctx.saved_tensors, dy.contiguous())

    torch.manual_seed(1)
    leaf = [t.requires_grad_() for t in (torch.randn(30, 136, device="cuda"),
                                         torch.rand(136, device="cuda") + 0.5,
                                         torch.randn(136, device="cuda"))]
    dy = torch.randn(30, 136, device="cuda")
    Norm.apply(*leaf).backward(dy)
    ref = [t.detach().double().requires_grad_() for t in leaf]
    torch.nn.functional.layer_norm(ref[0], (136,), ref[1], ref[2], 1e-5).backward(dy.double())
    for p, q in zip(leaf, ref):
        # sums of at most 136 terms, some 40 roundings of 2^-24 each, of the tensor's norm
        assert (p.grad.double() - q.grad).norm() <= 40 * 2.0 ** -24 * q.grad.norm()
