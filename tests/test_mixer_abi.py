"""Refusals of the mixer's entry points, on the host: bad arguments return a
status before anything is enqueued, and the binding refuses bad tensors."""
import ctypes
import math

import pytest
import torch

import gated_group_rmsnorm_gb300 as g
from gated_group_rmsnorm_gb300 import binding

# Fake "device" addresses, far apart: validation never dereferences them.
AT = {n: 0x100000000 * (i + 1) for i, n in enumerate(
    ("x", "dt", "b", "c", "a", "d", "dt_bias", "out", "state", "slots", "resume", "cu_seqlens",
     "workspace", "w", "bias"))}


def _conv(**kw):
    k = binding.ConvCall()
    base = dict(x=AT["x"], w=AT["w"], bias=AT["bias"], out=AT["out"], state=AT["state"],
                slots=AT["slots"], resume=AT["resume"], cu_seqlens=AT["cu_seqlens"], rows=8,
                seqs=2, width=16, x_row_stride=16, out_row_stride=16, state_slots=3,
                state_slot_stride=48, taps=4, activation=1, dtype=2)
    for n, v in {**base, **kw}.items():
        setattr(k, n, v)
    return k


def _scan(**kw):
    k = binding.ScanCall()
    base = dict(x=AT["x"], dt=AT["dt"], b=AT["b"], c=AT["c"], a=AT["a"], d=AT["d"],
                dt_bias=AT["dt_bias"], out=AT["out"], state=AT["state"], slots=AT["slots"],
                resume=AT["resume"], cu_seqlens=AT["cu_seqlens"], workspace=AT["workspace"],
                workspace_bytes=1 << 30, rows=8, seqs=2, heads=4, head_dim=8, groups=2,
                state_size=16, x_row_stride=32, dt_row_stride=4, b_row_stride=32, c_row_stride=32,
                out_row_stride=32, state_slots=3, state_slot_stride=512, dt_min=0.0,
                dt_max=math.inf, dt_softplus=1, dtype=2)
    for n, v in {**base, **kw}.items():
        setattr(k, n, v)
    return k


CONV_BAD = [
    (dict(rows=-1), binding.ERR_SHAPE),
    (dict(width=0), binding.ERR_SHAPE),
    (dict(seqs=0), binding.ERR_SHAPE),
    (dict(cu_seqlens=None, seqs=3), binding.ERR_SHAPE),      # 8 rows are not 3 equal sequences
    (dict(x_row_stride=15), binding.ERR_SHAPE),
    (dict(out_row_stride=15), binding.ERR_SHAPE),
    (dict(state_slot_stride=47), binding.ERR_SHAPE),
    (dict(slots=None, state_slots=1), binding.ERR_SHAPE),
    (dict(rows=1 << 40), binding.ERR_SHAPE),                 # offsets are 32-bit
    (dict(cu_seqlens=None, seqs=1, rows=1 << 60, x_row_stride=1 << 20), binding.ERR_SHAPE),
    (dict(taps=1), binding.ERR_UNSUPPORTED),
    (dict(taps=5), binding.ERR_UNSUPPORTED),
    (dict(dtype=3), binding.ERR_DTYPE),
    (dict(activation=2), binding.ERR_ARG),
    (dict(state=None, resume=None), binding.ERR_ARG),
    (dict(state=None, slots=None), binding.ERR_ARG),
    (dict(x=None), binding.ERR_NULL),
    (dict(out=None), binding.ERR_NULL),
    (dict(w=None), binding.ERR_NULL),
    (dict(x=AT["x"] + 1), binding.ERR_ALIGN),
    (dict(w=AT["w"] + 2), binding.ERR_ALIGN),
    (dict(cu_seqlens=AT["cu_seqlens"] + 2), binding.ERR_ALIGN),
    (dict(out=AT["x"] + 8), binding.ERR_OVERLAP),
    (dict(state=AT["x"] + 8), binding.ERR_OVERLAP),
    (dict(state=AT["out"] - 4), binding.ERR_OVERLAP),
    (dict(out=AT["w"]), binding.ERR_OVERLAP),
    (dict(out=AT["cu_seqlens"]), binding.ERR_OVERLAP),
    (dict(state=AT["slots"]), binding.ERR_OVERLAP),
]


@pytest.mark.parametrize("kw,status", CONV_BAD)
def test_conv_refuses(kw, status):
    assert g.load().ggrn_conv(ctypes.byref(_conv(**kw)), None) == status


SCAN_BAD = [
    (dict(rows=-1), binding.ERR_SHAPE),
    (dict(heads=0), binding.ERR_SHAPE),
    (dict(heads=3), binding.ERR_SHAPE),                      # not a multiple of the groups
    (dict(groups=0), binding.ERR_SHAPE),
    (dict(head_dim=0), binding.ERR_SHAPE),
    (dict(state_size=0), binding.ERR_SHAPE),
    (dict(state_size=257), binding.ERR_UNSUPPORTED),
    (dict(heads=65538), binding.ERR_UNSUPPORTED),
    (dict(cu_seqlens=None, seqs=3), binding.ERR_SHAPE),
    (dict(x_row_stride=31), binding.ERR_SHAPE),
    (dict(dt_row_stride=3), binding.ERR_SHAPE),
    (dict(b_row_stride=31), binding.ERR_SHAPE),
    (dict(c_row_stride=31), binding.ERR_SHAPE),
    (dict(out_row_stride=31), binding.ERR_SHAPE),
    (dict(state_slot_stride=511), binding.ERR_SHAPE),
    (dict(slots=None, state_slots=1), binding.ERR_SHAPE),
    (dict(dtype=-1), binding.ERR_DTYPE),
    (dict(dt_min=-1.0), binding.ERR_ARG),
    (dict(dt_min=2.0, dt_max=1.0), binding.ERR_ARG),
    (dict(dt_min=math.nan), binding.ERR_ARG),
    (dict(dt_max=math.nan), binding.ERR_ARG),
    (dict(state=None, slots=None), binding.ERR_ARG),
    (dict(a=None), binding.ERR_NULL),
    (dict(dt=None), binding.ERR_NULL),
    (dict(b=None), binding.ERR_NULL),
    (dict(out=None), binding.ERR_NULL),
    (dict(a=AT["a"] + 1), binding.ERR_ALIGN),
    (dict(state=AT["state"] + 2), binding.ERR_ALIGN),
    (dict(b=AT["b"] + 1), binding.ERR_ALIGN),
    (dict(out=AT["x"]), binding.ERR_OVERLAP),
    (dict(out=AT["dt"] + 2), binding.ERR_OVERLAP),
    (dict(state=AT["c"]), binding.ERR_OVERLAP),
    (dict(workspace=AT["out"]), binding.ERR_OVERLAP),
]


@pytest.mark.parametrize("kw,status", SCAN_BAD)
def test_scan_refuses(kw, status):
    assert g.load().ggrn_scan(ctypes.byref(_scan(**kw)), None) == status


def test_scan_refuses_a_missing_or_short_workspace():
    lib = g.load()
    # one long sequence of few heads has to be cut
    k = _scan(rows=1 << 16, seqs=1, x_row_stride=32)
    n = lib.ggrn_scan_workspace_bytes(ctypes.byref(k))
    assert n > 0
    k.workspace_bytes = n - 1
    assert lib.ggrn_scan(ctypes.byref(k), None) == binding.ERR_ARG
    k.workspace_bytes = n
    k.workspace = AT["workspace"] + 8
    assert lib.ggrn_scan(ctypes.byref(k), None) == binding.ERR_ALIGN
    k.workspace, k.workspace_bytes = None, 0
    assert lib.ggrn_scan(ctypes.byref(k), None) == binding.ERR_NULL


def test_workspace_bytes_of_invalid_and_short_calls():
    lib = g.load()
    assert lib.ggrn_scan_workspace_bytes(None) == 0
    assert lib.ggrn_scan_workspace_bytes(ctypes.byref(_scan(heads=3))) == 0
    assert lib.ggrn_scan_workspace_bytes(ctypes.byref(_scan())) == 0


def test_steps_refuse():
    lib = g.load()
    assert lib.ggrn_conv_step(ctypes.byref(_conv(state=None, slots=None)), None) == binding.ERR_NULL
    assert lib.ggrn_scan_step(ctypes.byref(_scan(state=None, slots=None)), None) == binding.ERR_NULL
    # 8 rows need 8 entries when no slots are given
    assert lib.ggrn_conv_step(ctypes.byref(_conv(slots=None)), None) == binding.ERR_SHAPE
    assert lib.ggrn_scan_step(ctypes.byref(_scan(slots=None)), None) == binding.ERR_SHAPE
    for f in (lib.ggrn_conv, lib.ggrn_conv_step, lib.ggrn_scan, lib.ggrn_scan_step):
        assert f(None, None) == binding.ERR_ARG


def test_nothing_to_do_is_fine():
    lib = g.load()
    none = dict(x=None, out=None, state=None, slots=None, resume=None)
    assert lib.ggrn_conv(ctypes.byref(_conv(rows=0, **none)), None) == binding.OK
    assert lib.ggrn_conv_step(ctypes.byref(_conv(rows=0, **none)), None) == binding.OK
    assert lib.ggrn_scan(ctypes.byref(_scan(rows=0, **none)), None) == binding.OK
    assert lib.ggrn_scan_step(ctypes.byref(_scan(rows=0, **none)), None) == binding.OK


def test_graph_of_steps_refuses():
    lib = g.load()
    handle = ctypes.c_void_p()
    steps = (binding.Step * 1)()
    steps[0].kind = 7
    assert lib.ggrn_graph_create_steps(steps, 1, ctypes.byref(handle)) == binding.ERR_ARG
    steps[0].kind = binding.STEP_CONV
    steps[0].u.conv = _conv(taps=9)
    assert lib.ggrn_graph_create_steps(steps, 1, ctypes.byref(handle)) == binding.ERR_UNSUPPORTED
    steps[0].kind = binding.STEP_SCAN
    steps[0].u.scan = _scan(heads=3)
    assert lib.ggrn_graph_create_steps(steps, 1, ctypes.byref(handle)) == binding.ERR_SHAPE
    assert lib.ggrn_graph_create_steps(None, 1, ctypes.byref(handle)) == binding.ERR_ARG


def test_binding_runs_on_cuda_only():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        g.causal_conv(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="CUDA"):
        g.causal_conv_step(x, torch.zeros(4, 3, 8), torch.zeros(8, 4))
    with pytest.raises(ValueError, match="CUDA"):
        g.ssm_scan(x, x, x, x, x, head_dim=8, state_size=8)
    with pytest.raises(ValueError, match="CUDA"):
        g.ssm_scan_step(x, x, x, x, x, torch.zeros(4, 1, 8, 8))


def test_rows_of_folds_leading_axes():
    t = torch.zeros(2, 3, 10)[:, :, 4:8]
    assert binding._rows_of(t, 4, "t") == (6, 10)
    assert binding._rows_of(torch.zeros(5, 7)[:, 3:4], 1, "t") == (5, 7)
    assert binding._rows_of(torch.zeros(2, 5, 7)[:, :, 6:7], 1, "t") == (10, 7)
    assert binding._rows_of(torch.zeros(1, 7)[:, 6:7], 1, "t") == (1, 1)
    assert binding._rows_of(torch.zeros(7, 50)[:, 3:7].unflatten(0, (7, 1)), 4, "t") == (7, 50)
    assert binding._rows_of(torch.zeros(3, 0, 7), 7, "t")[0] == 0
    with pytest.raises(ValueError):
        binding._rows_of(torch.zeros(4, 6, 7)[:, :3, 3:4], 1, "t")
    with pytest.raises(ValueError):
        binding._rows_of(torch.zeros(4, 6, 7)[:, :3], 7, "t")
