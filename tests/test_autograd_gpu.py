"""The operators and autograd: outputs carry no graph, the documentation says so, and
the backward passes serve a torch.autograd.Function."""
import pytest
import torch

import gated_group_rmsnorm_gb300 as g
from tests import train_ref as ref


def test_the_documentation_says_so():
    for f in (g.forward, g.backward, g.layer_norm, g.layer_norm_backward, g.linear_recurrence,
              g.linear_recurrence_step, g.linear_recurrence_backward):
        assert "autograd" in f.__doc__, f.__name__
    assert "autograd" in g.__doc__


def _leaves(*shape):
    gen = torch.Generator().manual_seed(0)
    return [torch.randn(*shape, generator=gen).cuda().requires_grad_() for _ in range(4)]


@pytest.mark.gpu
def test_outputs_carry_no_graph():
    x, i, r, dout = _leaves(70, 96)
    w = torch.ones(96, device="cuda").requires_grad_()
    a = (-w).detach().requires_grad_()
    state = torch.zeros(70, 96, device="cuda")
    got = [g.layer_norm(x, w, eps=1e-5), g.linear_recurrence(x, i, r, a),
           g.linear_recurrence_step(x, i, r, a, state),
           g.forward(x, i, w, group_size=32, eps=1e-5),
           *g.layer_norm_backward(dout, x, w, eps=1e-5),
           *g.backward(dout, x, i, w, group_size=32, eps=1e-5),
           *g.linear_recurrence_backward(dout, x, i, r, a)[:4]]
    assert not any(t.requires_grad or t.grad_fn is not None for t in got)


class Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, i, r, a):
        saved = g.linear_recurrence_saved(x)
        ctx.save_for_backward(x, i, r, a, saved)
        return g.linear_recurrence(x, i, r, a, saved=saved)

    @staticmethod
    def backward(ctx, dout):
        x, i, r, a, saved = ctx.saved_tensors
        return g.linear_recurrence_backward(dout, x, i, r, a, saved=saved)[:4]


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b):
        ctx.save_for_backward(x, w)
        return g.layer_norm(x, w, b, eps=1e-5)

    @staticmethod
    def backward(ctx, dout):
        return g.layer_norm_backward(dout.contiguous(), *ctx.saved_tensors, eps=1e-5)


@pytest.mark.gpu
def test_as_the_backward_of_a_function():
    x, i, r, dout = _leaves(150, 64)
    a = (-0.1 * torch.rand(64, generator=torch.Generator().manual_seed(1))).cuda().requires_grad_()
    w, b = (torch.ones(64, device="cuda").requires_grad_() for _ in range(2))
    dout = dout.detach()
    y = LayerNorm.apply(x, w, b)
    Recurrence.apply(y, i, r, a).backward(dout)
    want = ref.recur_backward(dout, y.detach(), i.detach(), r.detach(), a.detach(), [(0, 150)])
    for n, t in (("di", i), ("dr", r), ("da", a)):
        ref.assert_close(t.grad, *want[n], torch.float32, n)
    dy = g.linear_recurrence_backward(dout, y.detach(), i.detach(), r.detach(), a.detach())[0]
    want = ref.layer_norm_backward(dy, x.detach(), w.detach(), 1e-5)
    for n, t in (("dx", x), ("dw", w), ("db", b)):
        ref.assert_close(t.grad, *want[n], torch.float32, n)
