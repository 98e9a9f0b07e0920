"""The workspace of the scan: the size named for a call is enough for it."""
import pytest
import torch

import gated_group_rmsnorm_gb300 as g
from tests.test_scan_gpu import Case, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shift", [0, 1, 2, 4])
def test_workspace_bytes_for_a_given_out(shift):
    """The size named for a call is enough for it, wherever its out lies."""
    rows, heads, head_dim, state_size = 3000, 4, 64, 128
    k = Case(rows, heads, head_dim, 1, state_size, torch.bfloat16)
    v, w = k.on()
    width = heads * head_dim
    out = torch.zeros(rows * width + shift, dtype=torch.bfloat16,
                      device="cuda")[shift:].view(rows, width)
    n = g.scan_workspace_bytes(v["x"], v["dt"], w["a"], v["b"], v["c"], head_dim=head_dim,
                               state_size=state_size, out=out)
    assert n > 0
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    g.ssm_scan(v["x"], v["dt"], w["a"], v["b"], v["c"], head_dim=head_dim, state_size=state_size,
               d=w["d"], dt_bias=w["dt_bias"], out=out, workspace=ws)
    want, bound, size, *_ = k.want(spans=[(0, rows)])
    check(out, want, bound, size, torch.bfloat16)
    with pytest.raises(g.GgrnError):
        g.ssm_scan(v["x"], v["dt"], w["a"], v["b"], v["c"], head_dim=head_dim,
                   state_size=state_size, out=out, workspace=ws[:n - 16])


def test_asking_for_the_workspace_allocates_nothing():
    k = Case(3000, 4, 64, 1, 128, torch.bfloat16)
    v, w = k.on()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    assert g.scan_workspace_bytes(v["x"], v["dt"], w["a"], v["b"], v["c"], head_dim=64,
                                  state_size=128) > 0
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
