"""The scan of inputs that are not finite: each output and state entry is the
definition's infinity or NaN, whatever columns pad the state in the kernels.

All b, c and d here are positive and bounded away from zero and the decays are
slow, so that an infinity in x or dt makes infinities of one sign and nothing
underflows: a NaN can only come from a product with a padding zero, or from
another row, column or head.
"""
import math

import pytest
import torch

import gated_group_rmsnorm_gb300 as g
from tests import mixer_ref as ref
from tests.test_scan_gpu import DTYPES, Case

pytestmark = pytest.mark.gpu

# heads, head_dim, groups, state_size: state columns that fill no whole lane,
# vector, 16-column step or team, and some that do
SHAPES = [(2, 64, 1, 128), (2, 80, 2, 24), (1, 64, 1, 40), (3, 36, 1, 8), (2, 64, 1, 96),
          (2, 20, 1, 100), (2, 64, 1, 250), (1, 5, 1, 3), (2, 16, 1, 12), (1, 132, 1, 160)]


def _case(rows, shape, dtype, **kw):
    k = Case(rows, *shape, dtype, **kw)
    k.xbc = (k.xbc.float().abs() + 0.125).to(dtype)
    k.d = k.d.abs() + 0.125
    k.a = torch.full_like(k.a, -0.01)
    if k.state is not None:
        k.state = k.state.abs() + 0.125
    return k


def _kinds(t):
    """0 finite, 1 and -1 the infinities, 2 NaN."""
    t = t.double().cpu()
    return torch.where(torch.isnan(t), 2, torch.where(torch.isinf(t), t.sign().long(), 0))


def _same_kinds(got, want):
    assert torch.equal(_kinds(got), _kinds(want))


BAD = [("x", math.inf), ("x", -math.inf), ("x", math.nan), ("dt", math.inf)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("what,bad", BAD)
def test_prompts(dtype, shape, what, bad):
    rows = 300
    k = _case(rows, shape, dtype, slots=1, seed=5)
    k.views(k.xbc, k.z)[what][100, 0] = bad
    st = k.state.cuda()
    got = k.run(state=st)
    want, *_, new, _, _ = k.want(spans=[(0, rows)])
    _same_kinds(got, want)
    _same_kinds(st, new)
    assert (_kinds(want)[100:] != 0).any() and (_kinds(want)[:100] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_cut_prompt(dtype):
    rows, shape = 2000, (2, 64, 1, 24)
    k = _case(rows, shape, dtype, slots=1, seed=6)
    k.views(k.xbc, k.z)["x"][700, 3] = math.inf
    st = k.state.cuda()
    v, w = k.on()
    assert g.scan_workspace_bytes(v["x"], v["dt"], w["a"], v["b"], v["c"], head_dim=64,
                                  state_size=24) > 0
    got = k.run(state=st)
    want, *_, new, _, _ = k.want(spans=[(0, rows)])
    _same_kinds(got, want)
    _same_kinds(st, new)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("what,bad", BAD)
@pytest.mark.parametrize("shift", [0, 1])
def test_steps(dtype, shape, what, bad, shift):
    """shift: the pool at an address that leaves no vectors."""
    k = _case(3, shape, dtype, slots=3, seed=7)
    k.views(k.xbc, k.z)[what][1, 0] = bad
    pool = torch.zeros(k.state.numel() + shift, device="cuda")[shift:].view(k.state.shape)
    pool.copy_(k.state)
    v, w = k.on()
    got = g.ssm_scan_step(v["x"], v["dt"], w["a"], v["b"], v["c"], pool, d=w["d"],
                          dt_bias=w["dt_bias"])
    want, *_, new, _, _ = k.want(spans=[(i, i + 1) for i in range(3)], step=True)
    _same_kinds(got, want)
    _same_kinds(pool, new)
