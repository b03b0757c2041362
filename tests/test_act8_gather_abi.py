"""Refusals of mxfp8_dequantize_gather at the C ABI, before anything is launched (CPU only)."""
import ctypes
import os

from grouped_expert_gemm_amd import _lib

INV, UNS = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED
D, E8, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4104), ctypes.c_void_p(4097)


def test_refusals():
    if not os.path.exists(_lib.LIB_PATH):
        from grouped_expert_gemm_amd import build
        build.build()
    L = _lib.lib()

    def f(c=D, s=D, n=4, cols=64, src=D, rows=9, out=D):
        return L.mxfp8_dequantize_gather(c, s, n, cols, src, rows, out, None)

    assert f(n=-1) == INV and f(cols=-32) == INV and f(rows=-1) == INV and f(cols=40) == INV
    assert f(src=None) == INV and b"mxfp8_dequantize_gather" in L.moe_last_error()
    assert f(src=None, rows=4) == INV and b"NULL" in L.moe_last_error()     # no map, rows in their own order
    assert f(rows=1 << 31) == UNS and f(n=1 << 31) == UNS and f(cols=1 << 31) == UNS
    assert f(c=None) == INV and f(s=None) == INV and f(out=None) == INV
    assert f(c=E8) == INV and f(out=E8) == INV and f(src=ODD) == INV
    assert f(rows=0, src=None, n=0) == 0 and f(cols=0, c=None, s=None, out=None) == 0
