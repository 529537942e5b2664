"""The row operators' limits on both sides, through the size queries and the
host checks alone (no launch; fake pointers are never dereferenced)."""

import ctypes
import os

import pytest

import sparse_convolution_hash_amd.binding as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libspc.so not built")

P, BIG = ctypes.c_void_p(0x100000), 1 << 62
END = (1 << 31) - 4096


def norm(n, C, G, S):
    return B.lib().spc_group_norm_workspace(n, C, G, S, ctypes.byref(ctypes.c_size_t()))


def lr(n, C, S):
    return B.lib().spc_linear_recurrence_workspace(2, n, C, S, ctypes.byref(ctypes.c_size_t()), ctypes.byref(ctypes.c_size_t()))


def test_rows_and_samples():
    # beyond, row and sample numbers rounded up to tiles and waves pass 2^31
    assert norm(END - 1, 16, 1, 1) == norm(0, 16, 1, END - 1) == lr(END - 1, 16, 1) == lr(0, 16, END - 1) == B.SPC_OK
    for v in (END, END + 1, (1 << 31) - 2):
        assert norm(v, 16, 1, 1) == norm(0, 16, 1, v) == lr(v, 16, 1) == lr(0, 16, v) == B.SPC_ERR_ARG


def test_channels():
    C = 64 * 65535
    assert norm(1, C, 1, 1) == lr(1, C, 1) == B.SPC_OK
    assert norm(1, C + 16, 1, 1) == lr(1, C + 16, 1) == B.SPC_ERR_UNSUPPORTED


def test_threads_of_a_launch():
    # tiles of 512 rows x 64 channels: 2^24 workgroups of 256 threads are 2^32
    C, n = 4096, 1 << 27
    assert norm(n - 512, C, 64, 1) == lr(n - 512, C, 1) == B.SPC_OK
    assert norm(n, C, 64, 1) == lr(n, C, 1) == B.SPC_ERR_UNSUPPORTED
    L = B.lib()
    assert L.spc_group_norm_fwd(2, P, n, C, 64, None, 1, None, None, 1e-5, 0, None, P, P, P, BIG, None) == B.SPC_ERR_UNSUPPORTED
    assert L.spc_group_norm_bwd(2, P, P, n, C, 64, None, 1, None, None, P, 0, None, P, P, P, P, BIG, None) == B.SPC_ERR_UNSUPPORTED
    assert L.spc_linear_recurrence_fwd(2, P, P, C, n, C, None, 1, None, 0, None, P, None, None, P, BIG, None) == B.SPC_ERR_UNSUPPORTED
    # the step's threads take 8 elements
    assert L.spc_linear_recurrence_step(2, P, P, C, 1 << 23, C, P, P, P, None) == B.SPC_ERR_UNSUPPORTED


def test_groups():
    # any number below 2^31 (past 2^23 workgroups go over several each)
    for s in (1 << 18, 1 << 19, 1 << 22):
        assert norm(5000, 32, 32, s) == B.SPC_OK
    assert norm(5000, 32, 32, (1 << 26) - 2) == B.SPC_OK and norm(5000, 32, 32, 1 << 26) == B.SPC_ERR_UNSUPPORTED
