"""Shapes that the group norm's launches cannot take are refused on the host, before any device call."""
import ctypes

import pytest

from block_sparse_video_rearrange_b200 import rf

FAKE = [ctypes.c_void_p((i + 1) << 20) for i in range(9)]      # aligned, never dereferenced
LIB = rf.lib()


def desc(batch, groups, span):
    return rf.NormDesc(batch, 1, groups, 1, groups, groups, 1, groups, groups, 1, 0, 2, span, 0, 1e-5)


def workspace(d):
    out = ctypes.c_int64()
    return LIB.rf_group_norm_workspace_bytes(ctypes.byref(d), ctypes.byref(out)), out.value


@pytest.mark.parametrize("batch,groups", [(65535, 65535), (65535, 32769), (32769, 65535)])
def test_more_groups_than_a_grid_holds(batch, groups):
    d = desc(batch, groups, rf.SPANS["sample"])
    assert batch * groups >= 2 ** 31
    assert workspace(d)[0] == 6
    big = 1 << 50
    assert LIB.rf_group_norm(ctypes.byref(d), *FAKE[:6], big, None) == 6
    assert LIB.rf_group_norm_backward(ctypes.byref(d), *FAKE[:9], big, None) == 6


def test_what_a_grid_holds_is_taken():
    status, size = workspace(desc(65535, 32768, rf.SPANS["sample"]))
    assert status == 0 and size >= 65535 * 32768 * 8       # two means for each of them
    assert workspace(desc(65535, 65535, rf.SPANS["row"]))[0] == 0     # rows have no such grid
