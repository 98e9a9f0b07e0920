"""The bounded waits of the recurrence's clusters (GPU): a launch whose CTAs send
each other nothing makes every wait run out.  The kernel must end on its own,
report its bit in the device status word, write nothing, and leave the context
usable for the next call."""
import ctypes

import pytest
import torch

import gated_group_rmsnorm_gb300 as g
from gated_group_rmsnorm_gb300 import binding
from tests import train_ref as ref
from tests.test_recur_gpu import Case

pytestmark = pytest.mark.gpu


def _call(case, out):
    x, i, r = case.cuda()
    a = case.a.cuda()
    c = binding.RecurCall()
    for n, v in dict(x=x.data_ptr(), input_gate=i.data_ptr(), decay_gate=r.data_ptr(),
                     a=a.data_ptr(), out=out.data_ptr(), rows=case.rows, seqs=1, width=case.width,
                     x_row_stride=x.stride(0), input_gate_row_stride=i.stride(0),
                     decay_gate_row_stride=r.stride(0), out_row_stride=out.stride(0),
                     dtype=binding.DTYPE_CODE[case.dtype]).items():
        setattr(c, n, v)
    c.keep = (x, i, r, a)
    return c


@pytest.mark.parametrize("rows,dtype", [(1000, torch.bfloat16), (300, torch.float32)])
def test_waits_run_out_and_the_context_survives(rows, dtype):
    g.fault_status(clear=True)
    case = Case(rows, 128, dtype, 1)
    out = torch.full((rows, 128), 7.0, dtype=dtype, device="cuda")
    call = _call(case, out)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert g.load().ggrn_selftest_recur_timeout(ctypes.byref(call), stream) == binding.OK
    torch.cuda.synchronize()               # the kernel ended by itself
    assert g.fault_status(clear=True) == 128
    assert bool((out == 7.0).all())        # nothing written
    x, i, r = case.cuda()
    got = g.linear_recurrence(x, i, r, case.a.cuda())
    want, bound, *_ = ref.recur(*case.host(), case.a, [(0, rows)])
    ref.assert_close(got, want, bound, dtype)
    assert g.fault_status() == 0


def test_other_calls_are_refused():
    lib = g.load()
    case = Case(64, 128, torch.bfloat16, 1)  # one tile: no cluster
    out = torch.empty(64, 128, dtype=torch.bfloat16, device="cuda")
    call = _call(case, out)
    assert lib.ggrn_selftest_recur_timeout(ctypes.byref(call), None) == binding.ERR_UNSUPPORTED
    case = Case(300, 128, torch.bfloat16, 1)
    out = torch.empty(300, 128, dtype=torch.bfloat16, device="cuda")
    call, state = _call(case, out), torch.zeros(1, 128, device="cuda")
    call.state, call.state_slots, call.state_slot_stride = state.data_ptr(), 1, 128
    assert lib.ggrn_selftest_recur_timeout(ctypes.byref(call), None) == binding.ERR_UNSUPPORTED
    assert lib.ggrn_selftest_recur_timeout(None, None) == binding.ERR_ARG
