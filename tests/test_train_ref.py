"""The 64-bit references of the backward passes themselves: against torch's
differentiation of the definitions, and against differences."""
import pytest
import torch

from tests import train_ref as ref

SPANS = [(1, 1), (1, 2), (2, 9), (9, 9), (9, 30)]


def _near(got, want):
    assert torch.allclose(got, want, rtol=1e-9, atol=1e-11), float((got - want).abs().max())


def _recur_inputs(rows=33, width=6, seqs=5):
    gen = torch.Generator().manual_seed(3)
    x, ig, rg, dout = (torch.randn(rows, width, generator=gen, dtype=torch.float64)
                       for _ in range(4))
    a = -torch.rand(width, generator=gen, dtype=torch.float64) * torch.tensor(
        [0.01, 0.1, 0.3, 1.0, 4.0, 12.0], dtype=torch.float64)
    state = torch.randn(seqs, width, generator=gen, dtype=torch.float64)
    dstate = torch.randn(seqs, width, generator=gen, dtype=torch.float64)
    return x, ig, rg, dout, a, state, dstate


def _recur_loss(x, ig, rg, a, start, dout, dstate):
    p = a * torch.sigmoid(rg)
    e, b = torch.exp(p), torch.sqrt(-torch.expm1(2 * p)) * torch.sigmoid(ig) * x
    loss = 0
    for q, (r0, r1) in enumerate(SPANS):
        h = start[q]
        for t in range(r0, r1):
            h = e[t] * h + b[t]
            loss = loss + (h * dout[t]).sum()
        loss = loss + (h * dstate[q]).sum()
    return loss


def test_recurrence_against_differentiation_and_differences():
    x, ig, rg, dout, a, state, dstate = _recur_inputs()
    resume = torch.tensor([1, 0, 1, 1, 0], dtype=torch.bool)
    leaves = [t.clone().requires_grad_() for t in (x, ig, rg, a)]
    start = (state * resume[:, None]).requires_grad_()
    want = torch.autograd.grad(_recur_loss(*leaves, start, dout, dstate), leaves + [start])
    got = ref.recur_backward(dout, x, ig, rg, a, SPANS, state, None, resume, dstate)
    for n, w in zip(("dx", "di", "dr", "da"), want):
        _near(got[n][0], w)
    _near(got["dh"][0], want[4] * resume[:, None])
    for k, n in enumerate(("dx", "di", "dr", "da")):  # differences, in one direction each
        args = [x, ig, rg, a]
        gen = torch.Generator().manual_seed(k)
        way = torch.randn(args[k].shape, generator=gen, dtype=torch.float64) * args[k].abs()
        step = 1e-6
        ends = []
        for s in (step, -step):
            moved = list(args)
            moved[k] = args[k] + s * way
            ends.append(_recur_loss(*moved, state * resume[:, None], dout, dstate))
        slope = (ends[0] - ends[1]) / (2 * step)
        assert abs(slope - (way * got[n][0]).sum()) <= 1e-6 * (1 + abs(slope))


def test_layer_norm_against_differentiation():
    gen = torch.Generator().manual_seed(0)
    x, dout = (torch.randn(7, 33, generator=gen, dtype=torch.float64) for _ in range(2))
    w, b = (torch.randn(33, generator=gen, dtype=torch.float64) for _ in range(2))
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    out = torch.nn.functional.layer_norm(leaves[0], (33,), leaves[1], leaves[2], 1e-5)
    _near(ref.layer_norm(x, w, b, 1e-5)[0], out.detach())
    want = torch.autograd.grad(out, leaves, dout)
    got = ref.layer_norm_backward(dout, x, w, 1e-5)
    for n, v in zip(("dx", "dw", "db"), want):
        _near(got[n][0], v)


@pytest.mark.parametrize("mode", ["mamba2", "onnx"])
def test_gated_norm_against_differentiation(mode):
    gen = torch.Generator().manual_seed(0)
    y, z, dout = (torch.randn(7, 36, generator=gen, dtype=torch.float64) for _ in range(3))
    w = torch.randn(36 if mode == "mamba2" else 12, generator=gen, dtype=torch.float64)
    leaves = [t.clone().requires_grad_() for t in (y, z, w)]
    act = torch.nn.functional.silu(leaves[1])
    v = (leaves[0] * act if mode == "mamba2" else leaves[0]).unflatten(1, (3, 12))
    v = v * torch.rsqrt((v * v).mean(2, keepdim=True) + 1e-3)
    out = v.flatten(1) * leaves[2] if mode == "mamba2" else (v * leaves[2]).flatten(1) * act
    want = torch.autograd.grad(out, leaves, dout)
    got = ref.norm_backward(dout, y, z, w, 12, 1e-3, mode)
    for n, v in zip(("dy", "dgate", "dw"), want):
        _near(got[n][0], v)
