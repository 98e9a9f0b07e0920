"""Sizes that the mixer's entry points refuse, as ggrn.h names them: on the host,
before anything is enqueued."""
import ctypes

import pytest

import gated_group_rmsnorm_gb300 as g
from gated_group_rmsnorm_gb300 import binding
from tests.test_mixer_abi import _conv, _scan


@pytest.mark.parametrize("kw", [dict(heads=65536, groups=1, x_row_stride=1 << 20,
                                     out_row_stride=1 << 20, dt_row_stride=1 << 17),
                                dict(head_dim=65536, x_row_stride=1 << 20, out_row_stride=1 << 20),
                                dict(state_size=257, b_row_stride=1024, c_row_stride=1024)])
def test_scan_sizes(kw):
    k = _scan(state=None, slots=None, resume=None, **kw)
    assert g.load().ggrn_scan(ctypes.byref(k), None) == binding.ERR_UNSUPPORTED
    assert g.load().ggrn_scan_workspace_bytes(ctypes.byref(k)) == 0


def test_conv_columns():
    n = 4194240 + 1
    k = _conv(width=n, x_row_stride=n, out_row_stride=n, state=None, slots=None, resume=None)
    assert g.load().ggrn_conv(ctypes.byref(k), None) == binding.ERR_UNSUPPORTED


def test_workspace_of_many_sequences():
    """Longer parts, not a refusal: at most 65535 sequences of more than one."""
    entry = 4 * 8 * 16 * 4 + 4 * 4  # bytes of a part's state and decays
    for dtype in (0, 1, 2):
        for rows in (1 << 20, 1 << 26, (1 << 31) - 1):
            k = _scan(rows=rows, seqs=70000, dtype=dtype, state=None, slots=None, resume=None)
            n = g.load().ggrn_scan_workspace_bytes(ctypes.byref(k))
            assert 0 <= n <= 2 * 65535 * entry + 32


@pytest.mark.parametrize("kw", [dict(rows=1 << 40), dict(rows=(1 << 63) - 1), dict(rows=1 << 31),
                                dict(rows=1 << 20, seqs=0), dict(rows=-1), dict(seqs=-1),
                                dict(rows=1 << 20, seqs=1 << 31),
                                dict(rows=1 << 20, seqs=3, cu_seqlens=None),
                                dict(rows=(1 << 63) - 1, seqs=1, cu_seqlens=None)])
def test_no_workspace_for_rows_that_are_refused(kw):
    """Rows and sequences that the scan refuses have no size of a workspace."""
    k = _scan(state=None, slots=None, resume=None, **kw)
    assert g.load().ggrn_scan(ctypes.byref(k), None) == binding.ERR_SHAPE
    assert g.load().ggrn_scan_workspace_bytes(ctypes.byref(k)) == 0
