"""The bounded waits of the scan's tensor-core kernel (GPU): a launch whose
copies of b and c are left out makes every stage's wait run out.  The kernel must
end on its own, report its bit in the device status word, write nothing, and
leave the context usable for the next call."""
import ctypes

import pytest
import torch

import gated_group_rmsnorm_gb300 as g
from gated_group_rmsnorm_gb300 import binding
from tests.test_scan_gpu import Case, check

pytestmark = pytest.mark.gpu


def _call(k, out, **kw):
    v, w = k.on()
    c = binding.ScanCall()
    for name, value in dict(
            x=v["x"].data_ptr(), dt=v["dt"].data_ptr(), b=v["b"].data_ptr(), c=v["c"].data_ptr(),
            a=w["a"].data_ptr(), d=w["d"].data_ptr(), dt_bias=w["dt_bias"].data_ptr(),
            out=out.data_ptr(), rows=k.rows, seqs=1, heads=k.heads, head_dim=k.head_dim,
            groups=k.groups, state_size=k.state_size, x_row_stride=v["x"].stride(0),
            dt_row_stride=v["dt"].stride(0), b_row_stride=v["b"].stride(0),
            c_row_stride=v["c"].stride(0), out_row_stride=out.stride(0), dt_min=0.0,
            dt_max=float("inf"), dt_softplus=1, dtype=binding.BF16, **kw).items():
        setattr(c, name, value)
    c.keep = (v, w)
    return c


# a full chunk, a partial one, several
@pytest.mark.parametrize("rows,head_dim", [(128, 80), (37, 64), (300, 64)])
def test_waits_run_out_and_the_context_survives(rows, head_dim):
    g.fault_status(clear=True)
    k = Case(rows, 2, head_dim, 1, 128, torch.bfloat16)
    out = torch.full((rows, 2 * head_dim), 7.0, dtype=torch.bfloat16, device="cuda")
    call = _call(k, out)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert g.load().ggrn_selftest_scan_timeout(ctypes.byref(call), stream) == binding.OK
    torch.cuda.synchronize()               # the kernel ended by itself
    assert g.fault_status(clear=True) == 64
    assert bool((out == 7.0).all())        # nothing written
    got = k.run()                          # tensor memory is free again
    want, bound, size, *_ = k.want(spans=[(0, rows)])
    check(got, want, bound, size, torch.bfloat16)
    assert g.fault_status() == 0


def test_other_calls_are_refused():
    lib = g.load()
    for k in (Case(8, 2, 64, 1, 128, torch.bfloat16), Case(8, 2, 64, 1, 250, torch.bfloat16)):
        out = torch.empty(8, 128, dtype=torch.bfloat16, device="cuda")
        state = torch.zeros(1, 2, 64, k.state_size, device="cuda")
        kw = dict(state=state.data_ptr(), state_slots=1, state_slot_stride=state[0].numel())
        call = _call(k, out, **(kw if k.state_size == 128 else {}))
        assert lib.ggrn_selftest_scan_timeout(ctypes.byref(call), None) == binding.ERR_UNSUPPORTED
    assert lib.ggrn_selftest_scan_timeout(None, None) == binding.ERR_ARG
