"""The recurrence where clusters take several turns of whole tiles by 16-byte copies:
clusters of different sizes, both directions, against the definitions in 64 bits."""
import pytest
import torch

from tests import train_ref as ref
from tests.test_recur_gpu import RESUME, Case, _check

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


# (rows, width, type): more tiles than a cluster's eight CTAs twice over; wider rows
# leave fewer CTAs to a cluster
@pytest.mark.parametrize("rows,width,dtype", [
    (1100, 512, BF16), (1100, 512, F32), (1537, 64, F16), (1300, 1920, BF16), (1300, 2560, BF16),
    (1300, 2880, F16), (1300, 1280, F32), (1300, 3840, BF16), (1300, 6720, BF16),
    (1300, 7680, BF16)])
def test_one_sequence_over_several_turns(rows, width, dtype):
    case = Case(rows, width, dtype, 1, seed=width, rate=0.1)
    _check(case, [(0, rows)], None, case.state, None, [1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_fast_channels_beside_slow_ones(dtype):
    """One channel of 64 decays faster than the series reaches."""
    case = Case(1200, 512, dtype, 1, seed=1, rate=0.1)
    case.a[5::64] = -3.0
    _check(case, [(0, 1200)], None, case.state, None, [1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_packed_sequences_over_several_turns(dtype):
    cu = [0, 3, 640, 640, 1000, 1064, 1400]
    case = Case(1400, 1024, dtype, len(cu) - 1, seed=2, rate=0.1)
    _check(case, ref.ranges(1400, cu), cu, case.state, None, RESUME[:len(cu) - 1])
