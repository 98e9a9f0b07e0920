"""Scans of more sequences than a grid's third dimension holds."""
import pytest
import torch

from tests import mixer_ref as ref
from tests.test_scan_gpu import DTYPES, Case, check, check_state

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_long_one_among_66000(dtype):
    """Most of them empty, some of one to three rows, one long enough to be cut."""
    seqs, long = 66000, 700
    gen = torch.Generator().manual_seed(41)
    lens = torch.where(torch.rand(seqs, generator=gen) < 0.005,
                       torch.randint(1, 4, (seqs,), generator=gen), 0)
    lens[65990] = long
    cu = torch.cat([torch.zeros(1, dtype=torch.long), lens.cumsum(0)]).to(torch.int32)
    rows = int(cu[-1])
    k = Case(rows, 1, 16, 1, 16, dtype, slots=5, seed=42)
    slots = torch.full((seqs,), -1, dtype=torch.int32)
    filled = torch.nonzero(lens).flatten()
    slots[filled[[0, 3, 5]]] = torch.tensor([4, 0, 2], dtype=torch.int32)
    slots[65990], slots[65999] = 1, 3
    st = k.state.cuda()
    resume = torch.ones(seqs, dtype=torch.bool)
    out = k.run(cu_seqlens=cu.cuda(), state=st, slots=slots.cuda(), resume=resume.cuda())
    spans = ref.ranges(rows, cu.tolist())
    want, bound, size, new, nb, ns = k.want(spans=spans, slots=slots.tolist(),
                                            resume=[True] * seqs)
    check(out, want, bound, size, dtype)
    check_state(st, new, nb, ns)
