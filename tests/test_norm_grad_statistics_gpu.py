"""The norms' gradients take the mean square as the forward pass does: divided by
the group's size."""
import pytest
import torch

import gated_group_rmsnorm_gb300 as g

pytestmark = pytest.mark.gpu
GROUPS = [3, 41, 77, 82, 100, 119, 187, 213, 429, 717, 960, 1001, 2047, 5000, 7680, 18000]


@pytest.mark.parametrize("mode", ["mamba2", "onnx"])
@pytest.mark.parametrize("group", GROUPS)
def test_the_forward_passs_statistics(group, mode):
    """One row of f32 with weights and a gradient of 1: the weight's gradient is what the
    forward pass gives, bit for bit.  silu(40) is 40 in f32, and y of 1, 2, 3 leaves
    squares whose sum is exact in any order (units of 64, below 2^24 of them), so that
    nothing but the mean and its root can differ."""
    gen = torch.Generator().manual_seed(group)
    w, gate = torch.ones(group, device="cuda"), torch.full((1, group), 40.0, device="cuda")
    dout = torch.ones(1, group, device="cuda")
    for _ in range(8):
        y = torch.randint(1, 4, (1, group), generator=gen).float().cuda()
        out = g.forward(y, gate, w, group_size=group, eps=0.0, mode=mode)
        dw = g.backward(dout, y, gate, w, group_size=group, eps=0.0, mode=mode)[2]
        assert torch.equal(dw, out[0])
