"""The MXFP4 products' limit on rows (CPU only): a launch holds fewer than 2^32 threads, and the
kernels that lay the rows out for the 256-row tiles take one 256-thread workgroup for 8192 values.
Calls past it are refused before anything is enqueued, and so is the query of their workspace."""
import ctypes

import pytest

from grouped_expert_gemm_amd import _lib

D = ctypes.c_void_p(4096)
A, M = _lib.MOE_BF16, _lib.MOE_MXFP4
UNS = _lib.MOE_ERR_UNSUPPORTED
HUGE = 1 << 62


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(_lib.LIB_PATH):
        from grouped_expert_gemm_amd import build
        build.build()
    return _lib.lib()


@pytest.mark.parametrize("act", [A, M])
@pytest.mark.parametrize("R,K", [(1 << 24, 8192), ((1 << 29) + 8, 256), (0x7FFFFFFF, 256), ((1 << 25) - 7, 4096)])
def test_linear(L, act, R, K):
    tab = _lib.ptr_table([4096])[0]
    st = L.moe_grouped_linear_mxfp4(1, R, K, 256, act, D, D, tab, tab, D, D, D, HUGE, None)
    assert st == UNS and b"too many" in L.moe_last_error()
    n = ctypes.c_size_t()
    d = _lib.MlpDesc(1, K, 256, M, act, M, 0)
    assert L.moe_workspace_size(_lib.MOE_OP_LINEAR_MXFP4, ctypes.byref(d), R, 0, 0, 0, ctypes.byref(n)) == UNS


@pytest.mark.parametrize("wt", [A, M])
def test_mlp(L, wt):
    tab = _lib.ptr_table([4096, 4096])[0]
    for R, H, I in ((1 << 24, 8192, 256), ((1 << 29) + 8, 256, 256)):
        d = _lib.MlpDesc(2, H, I, M, A, wt, 0)
        n = ctypes.c_size_t()
        assert L.moe_workspace_size(_lib.MOE_OP_MLP_FWD, ctypes.byref(d), R, 0, 0, 0, ctypes.byref(n)) == UNS
        st = L.moe_grouped_mlp_fwd(ctypes.byref(d), R, D, D, tab, tab, tab, tab, D, D, D, None, None, D, HUGE, None)
        assert st == UNS and b"too many" in L.moe_last_error()


def test_the_most_rows_of_one_launch(L):
    n = ctypes.c_size_t()
    d = _lib.MlpDesc(1, 8192, 256, M, A, M, 0)
    R = (1 << 24) - 8
    assert L.moe_workspace_size(_lib.MOE_OP_LINEAR_MXFP4, ctypes.byref(d), R, 0, 0, 0, ctypes.byref(n)) == 0
    assert n.value >= R * (8192 // 2 + 8192 // 32)
    # rows of few values an expert are read as they are: no such limit (row kernel)
    d = _lib.MlpDesc(128, 8192, 256, M, A, M, 0)
    assert L.moe_workspace_size(_lib.MOE_OP_LINEAR_MXFP4, ctypes.byref(d), 128 * 64, 0, 0, 0, ctypes.byref(n)) == 0
