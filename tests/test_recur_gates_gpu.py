"""The recurrence's gates by themselves: sequences of one row, where an output is a
product of a few factors and so has a relative bound.

u = 2^-24, f32.  E = exp(-|z|) is good to 5 u: 4 u of the hardware's exponential (2^-22)
and a rounding.  The larger of sigmoid(z) and sigmoid(-z) is 1 / (1 + E): at most half of E's 5 u,
a rounding, and 1.1 u of one Newton step; the smaller is E times that: 5 u less what the
larger has of them, and 3.1 u: both below 8.2 u.  p = a r has 9.2 u, and exp(p) 9.2 |p| u and,
by the series (p > -1/4; s = exp(p) - 1 is good to 2.5 u by itself, 1 + s rounds once)
(2.5 |p| + 1) u, elsewhere 4 u (expf: 2 ulp).  1 - exp(2 p) = -s (2 + s): s to 11.7 u (p's
error counts at most once; expm1f: 1 ulp), two roundings, and m, its root, half of that and
1.1 u: 8 u.
"""
import pytest
import torch

import gated_group_rmsnorm_gb300 as g
from tests import train_ref as ref
from tests.mixer_ref import U, rounding

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
WIDTH = 256


def _rows(*columns):
    """[n, 1, WIDTH] of each on the GPU: n sequences of one row."""
    return [c.reshape(-1, 1, WIDTH).cuda() for c in columns]


def _within(got, want, relative, dtype):
    got, want = got.double().cpu().reshape(want.shape), want
    tol = relative * want.abs()
    if dtype != torch.float32:
        tol = tol + rounding(want, dtype) * (1 + 2.0 ** -8)
    worst = ((got - want).abs() / tol).max()
    assert bool(((got - want).abs() <= tol).all()), float(worst)


def _forward(x, i, r, a, h0=None):
    """The outputs of the prompt form and of the step form."""
    n = x.shape[0]
    pools = [torch.zeros(n, WIDTH, device="cuda") if h0 is None else h0.cuda() for _ in range(2)]
    resume = torch.ones(n, dtype=torch.bool, device="cuda")
    yield g.linear_recurrence(x, i, r, a, state=pools[0], resume=resume)
    yield g.linear_recurrence_step(x[:, 0], i[:, 0], r[:, 0], a, pools[1])


def test_input_gate_of_f32():
    """Decays of 4e-18 leave m = 1, and x = 1 the gate itself."""
    gen = torch.Generator().manual_seed(0)
    z = torch.rand(64, WIDTH, generator=gen) * 120 - 80
    x, i, r = _rows(torch.ones_like(z), z, torch.full_like(z, 20.0))
    a = torch.full((WIDTH,), -40.0, device="cuda")
    for out in _forward(x, i, r, a):
        _within(out, torch.sigmoid(z.double()), 8.2 * U, torch.float32)


def _decay_inputs():
    gen = torch.Generator().manual_seed(1)
    z = torch.rand(64, WIDTH, generator=gen) * 24 - 16
    a = -torch.exp(torch.rand(WIDTH, generator=gen) * 10 - 6)  # 0.0025 to 55
    return z, a, a.double() * torch.sigmoid(z.double())


def test_decay_of_f32():
    """x = 0 leaves exp(p) times the state."""
    z, a, p = _decay_inputs()
    h0 = 1 + torch.rand(z.shape, generator=torch.Generator().manual_seed(2))
    x, i, r = _rows(torch.zeros_like(z), z, z)
    near = torch.where(p > -0.25, 2.5 * p.abs() + 1, 4.0)
    for out in _forward(x, i, r, a.cuda(), h0):
        _within(out, torch.exp(p) * h0.double(), (9.2 * p.abs() + near + 1) * 1.01 * U, torch.float32)


def test_root_of_f32():
    """An input gate of 1 (40) and x = 1 leave m."""
    z, a, p = _decay_inputs()
    x, i, r = _rows(torch.ones_like(z), torch.full_like(z, 40.0), z)
    for out in _forward(x, i, r, a.cuda()):
        _within(out, torch.sqrt(-torch.expm1(2 * p)), 8 * U, torch.float32)


def _open(dtype):
    """Logits of open gates, from where 1 - sigmoid is 3e-4 to where it is 1e-7."""
    gen = torch.Generator().manual_seed(3)
    return (torch.rand(64, WIDTH, generator=gen) * 8 + 8).to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_of_an_open_input_gate(dtype):
    """m = 1, x = 1, dout = 1: di = i (1 - i).  f32: i (of an E below 3e-4) 2.1 u, 1 - i 8.2 u,
    m 1.1 u and four products.  16 bit: 1 - i has 1.7 |z| u of its argument's roundings
    (|z| <= 16), 4 u of the exponential, 2 u of the reciprocal and two roundings, i 3 u, and
    four products."""
    z = _open(dtype)
    one = torch.ones_like(z)
    x, i, r, dout = _rows(one, z, one * 20, one)
    a = torch.full((WIDTH,), -40.0, device="cuda")
    _, di, _, _, _ = g.linear_recurrence_backward(dout, x, i, r, a)
    zd = z.double()
    want = torch.sigmoid(zd) * torch.sigmoid(-zd)
    _within(di, want, (20 if dtype == torch.float32 else 64) * U, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_of_an_open_decay_gate(dtype):
    """x = 1, i = 1, dout = 1, no state: dr = -a e^2 / m r (1 - r), p near a = -1/2.  f32: e (twice)
    5.6 u, 1 / m 5.2 u, r 2.1 u, 1 - r 8.2 u and six products: below 64 u.  16 bit: e 8 u, 1 - e
    12 u of it, 1 / m 12 u, r 3 u, 1 - r 35 u and six products: below 128 u."""
    z = _open(dtype)
    one = torch.ones_like(z)
    x, i, r, dout = _rows(one, one * 40, z, one)
    a = torch.full((WIDTH,), -0.5)
    _, _, dr, _, _ = g.linear_recurrence_backward(dout, x, i, r, a.cuda())
    zd = z.double()
    p = a.double() * torch.sigmoid(zd)
    want = (-a.double() * torch.exp(2 * p) / torch.sqrt(-torch.expm1(2 * p)) * torch.sigmoid(zd) *
            torch.sigmoid(-zd))
    _within(dr, want, (64 if dtype == torch.float32 else 128) * U, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_closed_decay_gate_and_a_large_input(dtype):
    """x / m passes what f32 holds, r x / m does not: finite gradients."""
    rows, width = 70, 96
    gen = torch.Generator().manual_seed(4)
    x = (torch.randn(rows, width, generator=gen) * 2.0 ** 90).to(dtype)
    i, dout = (torch.randn(rows, width, generator=gen).to(dtype) for _ in range(2))
    r = (torch.rand(rows, width, generator=gen) * 20 - 65).to(dtype)
    a = -0.1 * torch.rand(width, generator=gen) - 0.01
    want = ref.recur_backward(dout, x, i, r, a, [(0, rows)])
    got = g.linear_recurrence_backward(dout.cuda(), x.cuda(), i.cuda(), r.cuda(), a.cuda())
    for n, v in zip(("dx", "di", "dr", "da"), got):
        assert torch.isfinite(v).all(), n
        ref.assert_close(v, *want[n], torch.float32 if n == "da" else dtype, n)
