"""CPU checks of what the target side's plans promise: workgroups and workspaces
(256 compute units, as without a GPU or on the one it is built for)."""
import ctypes

import pytest

import draft_selection_topk16_amd as df2
from draft_selection_topk16_amd.binding import PagedKv, VerifyDims

F32, BF16 = 0, 1


def kv(B, N, Hq, Hkv, D, dtype, page=16, width=8192):
    at = 0x10000        # never dereferenced
    return PagedKv(at, at, at, at, at, Hkv * page * D, width, B, N, Hq, Hkv, D, page, 10, width, dtype)


def workspace(k, max_len=0):
    return df2.load().dflash2_paged_attention_workspace(ctypes.byref(k), max_len)


def parts(wgs, bm, D):
    """Bytes of two parts of bm rows of D outputs, a maximum and a sum a workgroup, and
    of its boundary's words."""
    return (2 * wgs * bm * D + (4 * bm + 8) * wgs) * 4


@pytest.mark.parametrize("dtype,D,n,bm,per_cu", [
    (BF16, 64, 8, 32, 2), (BF16, 64, 16, 64, 2), (BF16, 64, 32, 128, 2), (BF16, 64, 64, 256, 1),
    (BF16, 128, 8, 32, 1), (BF16, 128, 16, 64, 2), (BF16, 128, 32, 128, 2), (BF16, 128, 64, 256, 1),
    (BF16, 256, 8, 32, 1), (BF16, 256, 16, 64, 1), (BF16, 256, 32, 128, 1),
    (F32, 64, 8, 32, 1), (F32, 64, 32, 128, 2), (F32, 128, 8, 32, 1), (F32, 128, 32, 128, 1), (F32, 256, 8, 128, 1),
])
def test_no_more_stretches_than_workgroups_that_run_at_once(dtype, D, n, bm, per_cu):
    """By LDS: two stages of keys and values.  By registers: heads of 512 bytes and more
    leave one wave a SIMD, so one workgroup of four waves a compute unit."""
    assert workspace(kv(4, 4 * n, 32, 8, D, dtype)) == parts(256 * per_cu, bm, D)


def test_sizes_beyond_a_launch_are_refused():
    """A launch takes fewer than 2^32 threads: these sizes, small enough for memory,
    would need more."""
    lib, at = df2.load(), 0x100000
    k = kv(1, (1 << 26) - 3, 1, 1, 64, BF16)
    assert lib.dflash2_kv_append(ctypes.byref(k), None, 0, at, 64, at, 64, None, None, 1e-6, None, 0, 0, None, 0, None) == 2
    assert b"2^26" in lib.dflash2_last_error()
    for B, P in ((1 << 23, 1), (1 << 21, 7)):
        d = VerifyDims(B, P, 8, 1, BF16, 0)
        assert lib.dflash2_verify_workspace(ctypes.byref(d)) == 0
        assert lib.dflash2_verify(ctypes.byref(d), at, at, at, at, None, 1.0, at, at, at, at, at, 1 << 40, None) == 2
        assert b"too large" in lib.dflash2_last_error()
        assert lib.dflash2_verify_workspace(ctypes.byref(VerifyDims(B - 1, P, 8, 1, BF16, 0))) > 0
    assert lib.dflash2_draft_rows(at, at, at, 1 << 20, 64, 1, 1.0, at, None) == 2
    assert b"too many" in lib.dflash2_last_error()
