"""Prompts of the scan with many values in x that are not finite: the results
are the definition's, and no bounded wait of the kernels runs out over them."""
import math

import pytest
import torch

import gated_group_rmsnorm_gb300 as g
from tests.test_scan_gpu import DTYPES
from tests.test_scan_infinities_gpu import _case, _same_kinds

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
def test_an_infinity_beside_a_nan_of_its_column(dtype):
    """A NaN in an earlier chunk stays a NaN where an infinity joins it later."""
    rows, shape = 300, (1, 64, 1, 32)
    k = _case(rows, shape, dtype, slots=1, seed=8)
    x = k.views(k.xbc, k.z)["x"]
    x[20, 3], x[150, 3], x[150, 9] = math.nan, math.inf, -math.inf
    x[151, 9] = math.inf
    st = k.state.cuda()
    got = k.run(state=st)
    want, *_, new, _, _ = k.want(spans=[(0, rows)])
    _same_kinds(got, want)
    _same_kinds(st, new)


FILLS = {
    "nan": lambda t, gen: t.fill_(math.nan),
    "inf": lambda t, gen: t.fill_(math.inf),
    "-inf": lambda t, gen: t.fill_(-math.inf),
    "both": lambda t, gen: t.copy_(torch.where(torch.rand(t.shape, generator=gen) < 0.5, math.inf,
                                               -math.inf)),
    "some": lambda t, gen: t.copy_(torch.where(torch.rand(t.shape, generator=gen) < 0.02, math.inf,
                                               t.float())),
}


@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(2, 80, 1, 128), (2, 64, 2, 24), (1, 84, 1, 40)])
def test_x_full_of_them(dtype, shape, fill):
    """Three chunks and a bit; the first rows stay finite."""
    rows = 390
    k = _case(rows, shape, dtype, slots=1, seed=9)
    FILLS[fill](k.views(k.xbc, k.z)["x"][20:], torch.Generator().manual_seed(1))
    st = k.state.cuda()
    got = k.run(state=st)
    want, *_, new, _, _ = k.want(spans=[(0, rows)])
    _same_kinds(got, want)
    _same_kinds(st, new)
    assert g.fault_status() == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_b_and_c_of_both_signs(dtype):
    """Infinities that cancel: NaN from the definition's own sums."""
    rows, shape = 300, (2, 64, 1, 24)
    k = _case(rows, shape, dtype, slots=1, seed=10)
    v = k.views(k.xbc, k.z)
    v["b"][:, ::2] *= -1
    v["x"][130:, ::3] = math.inf
    st = k.state.cuda()
    got = k.run(state=st)
    want, *_, new, _, _ = k.want(spans=[(0, rows)])
    _same_kinds(got, want)
    _same_kinds(st, new)
    assert g.fault_status() == 0


def test_a_long_prompt_of_infinities():
    """The slowest case of the tensor-core kernel: infinities of one sign in
    every place of 2048 rows of each of several heads."""
    rows, heads, head_dim = 2048, 8, 80
    k = _case(rows, (heads, head_dim, 1, 128), torch.bfloat16, seed=11)
    k.a = torch.full_like(k.a, -0.001)
    k.views(k.xbc, k.z)["x"].fill_(math.inf)
    got = k.run()
    assert torch.isposinf(got).all()
    assert g.fault_status() == 0


@pytest.mark.parametrize("rows,row", [(1, 0), (40, 0), (300, 37), (300, 140)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_x_and_dt_of_one_row(dtype, rows, row):
    """An infinite dt beside x that are infinities of both signs, NaN and finite."""
    k = _case(rows, (2, 80, 1, 24), dtype, slots=1, seed=12)
    v = k.views(k.xbc, k.z)
    v["dt"][row, 0] = math.inf
    for col, bad in ((3, math.inf), (4, -math.inf), (9, math.nan), (85, math.inf)):
        v["x"][row, col] = bad
    st = k.state.cuda()
    got = k.run(state=st, resume=torch.ones(1, dtype=torch.bool).cuda())
    want, *_, new, _, _ = k.want(spans=[(0, rows)], resume=[True])
    _same_kinds(got, want)
    _same_kinds(st, new)
    assert g.fault_status() == 0
