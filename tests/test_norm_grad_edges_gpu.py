"""The gated norm's gradients at places of their own: teams of a CTA that hold no
group, and the statistics that the forward pass takes."""
import pytest
import torch

import gated_group_rmsnorm_gb300 as g
from tests import train_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("rows,groups,group", [(5, 17, 128), (4, 13, 77), (300, 17, 128),
                                               (1, 257, 8)])
def test_onnx_without_eps_where_teams_are_left_over(rows, groups, group, dtype):
    """A team that holds no group reads zeros, whose 1 / rms is infinite without eps:
    nothing of it reaches the scale's gradient."""
    gen = torch.Generator().manual_seed(groups)
    dout, y, z = (torch.randn(rows, groups * group, generator=gen).to(dtype) for _ in range(3))
    w = (1 + 0.5 * torch.randn(group, generator=gen)).to(dtype)
    want = ref.norm_backward(dout, y, z, w, group, 0.0, "onnx")
    got = g.backward(dout.cuda(), y.cuda(), z.cuda(), w.cuda(), group_size=group, eps=0.0,
                     mode="onnx")
    for n, v in zip(("dy", "dgate", "dw"), got):
        assert torch.isfinite(v).all(), n
        ref.assert_close(v, *want[n], torch.float32 if n == "dw" else dtype, n)
