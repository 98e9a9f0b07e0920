"""Refusals of the recurrence, layer norm and the backward passes, on the host: bad
arguments return a status before anything is enqueued, and the binding refuses bad
tensors."""
import ctypes

import pytest
import torch

import gated_group_rmsnorm_gb300 as g
from gated_group_rmsnorm_gb300 import binding
from gated_group_rmsnorm_gb300.binding import (ERR_ALIGN, ERR_ARG, ERR_DTYPE, ERR_NULL, ERR_OVERLAP,
                                               ERR_SHAPE, ERR_UNSUPPORTED, OK)

# Fake "device" addresses, far apart: validation never dereferences them.
AT = {n: 0x100000000 * (k + 1) for k, n in enumerate(
    ("x", "input_gate", "decay_gate", "a", "out", "state", "slots", "resume", "cu_seqlens", "saved",
     "dout", "dx", "dinput_gate", "ddecay_gate", "da", "dinitial", "dstate", "workspace", "w", "b",
     "dw", "db", "y", "gate", "dy", "dgate"))}
ROWS, WIDTH = 200, 32


def _make(cls, base, kw):
    k = cls()
    for n, v in {**{n: AT[n] for n, _ in cls._fields_ if n in AT}, **base, **kw}.items():
        setattr(k, n, v)
    return ctypes.byref(k)


def _strides(cls):
    return {n: WIDTH for n, _ in cls._fields_ if n.endswith("row_stride")}


def _recur(**kw):
    return _make(binding.RecurCall, dict(_strides(binding.RecurCall), rows=ROWS, seqs=2, width=WIDTH,
                                         state_slots=3, state_slot_stride=WIDTH, dtype=2), kw)


def _recur_backward(**kw):
    return _make(binding.RecurBackwardCall,
                 dict(_strides(binding.RecurBackwardCall), rows=ROWS, seqs=2, width=WIDTH,
                      state_slots=3, state_slot_stride=WIDTH, dtype=2, workspace_bytes=1 << 30), kw)


SEQS_BAD = [
    (dict(rows=-1), ERR_SHAPE),
    (dict(width=0), ERR_SHAPE),
    (dict(width=2097121, x_row_stride=1 << 22, state_slot_stride=1 << 22), ERR_UNSUPPORTED),
    (dict(seqs=0), ERR_SHAPE),
    (dict(cu_seqlens=None, seqs=3), ERR_SHAPE),
    (dict(rows=1 << 40), ERR_SHAPE),
    (dict(x_row_stride=WIDTH - 1), ERR_SHAPE),
    (dict(input_gate_row_stride=WIDTH - 1), ERR_SHAPE),
    (dict(decay_gate_row_stride=WIDTH - 1), ERR_SHAPE),
    (dict(state_slot_stride=WIDTH - 1), ERR_SHAPE),
    (dict(slots=None, state_slots=1), ERR_SHAPE),
    (dict(dtype=3), ERR_DTYPE),
    (dict(state=None, resume=None), ERR_ARG),
    (dict(state=None, slots=None), ERR_ARG),
    (dict(x=None), ERR_NULL),
    (dict(input_gate=None), ERR_NULL),
    (dict(decay_gate=None), ERR_NULL),
    (dict(a=None), ERR_NULL),
    (dict(x=AT["x"] + 1), ERR_ALIGN),
    (dict(a=AT["a"] + 2), ERR_ALIGN),
    (dict(state=AT["state"] + 2), ERR_ALIGN),
    (dict(saved=AT["saved"] + 2), ERR_ALIGN),
    (dict(cu_seqlens=AT["cu_seqlens"] + 2), ERR_ALIGN),
]
RECUR_BAD = SEQS_BAD + [
    (dict(out=None), ERR_NULL),
    (dict(out_row_stride=WIDTH - 1), ERR_SHAPE),
    (dict(out=AT["x"]), ERR_OVERLAP),
    (dict(out=AT["state"]), ERR_OVERLAP),
    (dict(state=AT["decay_gate"]), ERR_OVERLAP),
    (dict(saved=AT["out"] + 4), ERR_OVERLAP),
    (dict(saved=AT["state"]), ERR_OVERLAP),
    (dict(state=AT["slots"]), ERR_OVERLAP),
]
BACKWARD_BAD = SEQS_BAD + [
    (dict(dout=None), ERR_NULL),
    (dict(dx=None), ERR_NULL),
    (dict(dinput_gate=None), ERR_NULL),
    (dict(ddecay_gate=None), ERR_NULL),
    (dict(da=None), ERR_NULL),
    (dict(dout_row_stride=WIDTH - 1), ERR_SHAPE),
    (dict(ddecay_gate_row_stride=WIDTH - 1), ERR_SHAPE),
    (dict(da=AT["da"] + 1), ERR_ALIGN),
    (dict(dstate=AT["dstate"] + 1), ERR_ALIGN),
    (dict(dx=AT["dout"]), ERR_OVERLAP),
    (dict(dx=AT["dinput_gate"] + 64), ERR_OVERLAP),
    (dict(da=AT["a"]), ERR_OVERLAP),
    (dict(dinitial=AT["dstate"]), ERR_OVERLAP),
    (dict(dinitial=AT["state"]), ERR_OVERLAP),
    (dict(dx=AT["saved"]), ERR_OVERLAP),
]


@pytest.mark.parametrize("kw,status", RECUR_BAD)
def test_recurrence_refuses(kw, status):
    assert g.load().ggrn_recur(_recur(**kw), None) == status


@pytest.mark.parametrize("kw,status", BACKWARD_BAD)
def test_recurrence_backward_refuses(kw, status):
    assert g.load().ggrn_recur_backward(_recur_backward(**kw), None) == status


def test_recurrence_step_refuses():
    lib = g.load()
    assert lib.ggrn_recur_step(_recur(state=None, slots=None), None) == ERR_NULL
    assert lib.ggrn_recur_step(_recur(slots=None), None) == ERR_SHAPE  # 200 rows, 3 entries
    for f in (lib.ggrn_recur, lib.ggrn_recur_step, lib.ggrn_recur_backward):
        assert f(None, None) == ERR_ARG


def test_recurrence_workspace():
    """Without the kept states the backward pass needs room for them."""
    lib = g.load()
    need = lib.ggrn_recur_backward_workspace_bytes(_recur_backward(saved=None))
    assert need >= 4 * 4 * WIDTH  # 200 rows: four states
    for kw, status in ((dict(workspace=None), ERR_NULL), (dict(workspace_bytes=need - 1), ERR_ARG),
                       (dict(workspace=AT["workspace"] + 8), ERR_ALIGN),
                       (dict(workspace=AT["dx"]), ERR_OVERLAP)):
        assert lib.ggrn_recur_backward(_recur_backward(saved=None, **kw), None) == status
    assert lib.ggrn_recur_backward_workspace_bytes(None) == 0
    assert lib.ggrn_recur_backward_workspace_bytes(_recur_backward(dtype=7)) == 0
    assert lib.ggrn_recur_backward_workspace_bytes(_recur_backward(seqs=0)) == 0


def test_columns_beside_each_other_are_no_overlap():
    """The same rows, columns beside each other: refused only where they meet."""
    lib = g.load()

    def overlap(apart, out_stride, stride=3 * WIDTH):
        k = binding.LayerNormCall()
        for n, v in dict(x=AT["x"], w=AT["w"], b=AT["b"], out=AT["x"] + 2 * apart, rows=ROWS, width=WIDTH,
                         x_row_stride=stride, out_row_stride=out_stride, eps=1e-5, dtype=2).items():
            setattr(k, n, v)
        steps = (binding.Step * 2)()
        steps[0].kind = binding.STEP_LAYER_NORM
        steps[0].u.layer_norm = k
        steps[1].kind = 99  # (refused: nothing is captured)
        return lib.ggrn_graph_create_steps(steps, 2, ctypes.byref(ctypes.c_void_p()))

    s = 3 * WIDTH
    assert overlap(WIDTH, s) == ERR_ARG            # beside x: the next step is what is refused
    assert overlap(2 * WIDTH, s) == ERR_ARG
    assert overlap(WIDTH - 1, s) == ERR_OVERLAP
    assert overlap(2 * WIDTH + 1, s) == ERR_OVERLAP
    assert overlap(0, s) == ERR_OVERLAP
    assert overlap(WIDTH, s + 1) == ERR_OVERLAP    # rows of another stride drift into each other
    assert overlap(s * 5 + WIDTH, s) == ERR_ARG    # from a later row on


def _layer_norm(**kw):
    return _make(binding.LayerNormCall, dict(_strides(binding.LayerNormCall), rows=ROWS, width=WIDTH,
                                             eps=1e-5, dtype=2), kw)


def _layer_norm_backward(**kw):
    return _make(binding.LayerNormBackwardCall,
                 dict(_strides(binding.LayerNormBackwardCall), rows=ROWS, width=WIDTH, eps=1e-5,
                      dtype=2, workspace_bytes=1 << 30), kw)


def _backward(**kw):
    return _make(binding.BackwardCall, dict(_strides(binding.BackwardCall), rows=ROWS, width=WIDTH,
                                            group_size=8, eps=1e-5, dtype=2, mode=0,
                                            workspace_bytes=1 << 30), kw)


LN_BAD = [
    (dict(rows=-1), ERR_SHAPE),
    (dict(width=0), ERR_SHAPE),
    (dict(x_row_stride=WIDTH - 1), ERR_SHAPE),
    (dict(rows=1 << 61, x_row_stride=1 << 20), ERR_SHAPE),
    (dict(dtype=-1), ERR_DTYPE),
    (dict(x=None), ERR_NULL),
    (dict(w=None), ERR_NULL),
    (dict(x=AT["x"] + 1), ERR_ALIGN),
    (dict(w=AT["w"] + 2), ERR_ALIGN),
]


@pytest.mark.parametrize("kw,status", LN_BAD + [
    (dict(out=None), ERR_NULL), (dict(out_row_stride=WIDTH - 1), ERR_SHAPE),
    (dict(b=AT["b"] + 1), ERR_ALIGN), (dict(out=AT["x"] + 64), ERR_OVERLAP),
    (dict(out=AT["w"]), ERR_OVERLAP), (dict(out=AT["b"]), ERR_OVERLAP)])
def test_layer_norm_refuses(kw, status):
    assert g.load().ggrn_layer_norm(_layer_norm(**kw), None) == status


@pytest.mark.parametrize("kw,status", LN_BAD + [
    (dict(dout=None), ERR_NULL), (dict(dx=None), ERR_NULL), (dict(dw=None), ERR_NULL),
    (dict(dout_row_stride=WIDTH - 1), ERR_SHAPE), (dict(dx_row_stride=WIDTH - 1), ERR_SHAPE),
    (dict(db=AT["db"] + 2), ERR_ALIGN), (dict(dx=AT["dout"]), ERR_OVERLAP),
    (dict(dw=AT["db"]), ERR_OVERLAP), (dict(dx=AT["dw"]), ERR_OVERLAP),
    (dict(workspace=None), ERR_NULL), (dict(workspace=AT["workspace"] + 4), ERR_ALIGN),
    (dict(workspace_bytes=64), ERR_ARG), (dict(workspace=AT["x"]), ERR_OVERLAP)])
def test_layer_norm_backward_refuses(kw, status):
    assert g.load().ggrn_layer_norm_backward(_layer_norm_backward(**kw), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), ERR_SHAPE), (dict(group_size=0), ERR_SHAPE), (dict(group_size=5), ERR_SHAPE),
    (dict(mode=2), ERR_DTYPE), (dict(mode=1), ERR_DTYPE),  # ONNX has no bf16
    (dict(dtype=5), ERR_DTYPE), (dict(gate_row_stride=WIDTH - 1), ERR_SHAPE),
    (dict(y=None), ERR_NULL), (dict(gate=None), ERR_NULL), (dict(dgate=None), ERR_NULL),
    (dict(w=None), ERR_NULL), (dict(dw=None), ERR_NULL), (dict(dy=AT["dy"] + 1), ERR_ALIGN),
    (dict(dy=AT["y"]), ERR_OVERLAP), (dict(dy=AT["dgate"]), ERR_OVERLAP),
    (dict(dgate=AT["dout"]), ERR_OVERLAP), (dict(dw=AT["w"]), ERR_OVERLAP),
    (dict(workspace=None), ERR_NULL), (dict(workspace_bytes=64), ERR_ARG),
    (dict(workspace=AT["dgate"]), ERR_OVERLAP),
    (dict(width=65536 * 64, group_size=64, **{n: 65536 * 64 for n in _strides(binding.BackwardCall)}),
     ERR_UNSUPPORTED)])
def test_backward_refuses(kw, status):
    assert g.load().ggrn_backward(_backward(**kw), None) == status


def test_workspaces_of_invalid_calls():
    lib = g.load()
    assert lib.ggrn_layer_norm_backward_workspace_bytes(None) == 0
    assert lib.ggrn_layer_norm_backward_workspace_bytes(_layer_norm_backward(width=0)) == 0
    assert lib.ggrn_layer_norm_backward_workspace_bytes(_layer_norm_backward(rows=0)) == 0
    assert lib.ggrn_backward_workspace_bytes(_backward(group_size=5)) == 0
    assert lib.ggrn_backward_workspace_bytes(_backward(mode=3)) == 0
    for f in (lib.ggrn_layer_norm, lib.ggrn_layer_norm_backward, lib.ggrn_backward):
        assert f(None, None) == ERR_ARG


def test_nothing_to_do_is_fine():
    lib = g.load()
    none = dict(x=None, input_gate=None, decay_gate=None, out=None, state=None, slots=None,
                resume=None)
    assert lib.ggrn_recur(_recur(rows=0, **none), None) == OK
    assert lib.ggrn_recur_step(_recur(rows=0, **none), None) == OK
    assert lib.ggrn_layer_norm(_layer_norm(rows=0, x=None, out=None, w=None), None) == OK


def test_graph_of_steps_refuses():
    lib = g.load()
    handle = ctypes.c_void_p()
    steps = (binding.Step * 1)()
    steps[0].kind = binding.STEP_RECUR
    steps[0].u.recur = _recur(state=None, slots=None)._obj
    assert lib.ggrn_graph_create_steps(steps, 1, ctypes.byref(handle)) == ERR_NULL
    steps[0].kind = binding.STEP_LAYER_NORM
    steps[0].u.layer_norm = _layer_norm(w=None)._obj
    assert lib.ggrn_graph_create_steps(steps, 1, ctypes.byref(handle)) == ERR_NULL


def test_binding_runs_on_cuda_only():
    x, v = torch.zeros(4, 8), torch.zeros(8)
    for call in (lambda: g.linear_recurrence(x, x, x, v),
                 lambda: g.linear_recurrence_step(x, x, x, v, torch.zeros(4, 8)),
                 lambda: g.linear_recurrence_backward(x, x, x, x, v),
                 lambda: g.layer_norm(x, v, eps=1e-5),
                 lambda: g.layer_norm_backward(x, x, v, eps=1e-5),
                 lambda: g.backward(x, x, x, v, group_size=8, eps=1e-5)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for call in (lambda: g.linear_recurrence(None, x, x, v), lambda: g.layer_norm(3, v, eps=1e-5)):
        with pytest.raises(ValueError, match="tensor"):
            call()


def test_saved_has_a_state_for_every_64_rows():
    for rows, n in ((0, 0), (1, 1), (64, 1), (65, 2), (1000, 16)):
        t = g.linear_recurrence_saved(torch.zeros(rows, 10, dtype=torch.bfloat16))
        assert t.shape == (n, 10) and t.dtype == torch.float32
    assert g.linear_recurrence_saved(torch.zeros(3, 50, 10)).shape == (3, 10)
    assert binding.SAVED_ROWS == 64
