"""Refusals of the balance loss and the norms at the C ABI, before anything is launched
(CPU only), and their workspace sizes."""
import ctypes

import pytest

from grouped_expert_gemm_amd import _lib

INV, UNS, WS = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE
D = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4097)


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(_lib.LIB_PATH):
        from grouped_expert_gemm_amd import build
        build.build()
    return _lib.lib()


def _size(L, op, desc, R, T, E, k):
    n = ctypes.c_size_t()
    st = L.moe_workspace_size(op, ctypes.byref(desc) if desc else None, R, T, E, k, ctypes.byref(n))
    return st, n.value


def test_balance_loss(L):
    def fwd(logits=D, idx=D, T=64, E=8, k=2, seq=32, counts=D, tokens=D, loss=D, ws=D, nbytes=1 << 20):
        return L.moe_balance_loss(logits, idx, None, T, E, k, seq, 1.0, 0.0, counts, tokens, loss, ws, nbytes, None)

    assert fwd(T=-1) == INV and fwd(E=0) == INV and fwd(E=257) == INV and fwd(k=0) == INV and fwd(k=9) == INV
    assert fwd(seq=0) == INV and fwd(seq=63) == INV and b"seq_len" in L.moe_last_error()
    assert fwd(T=1 << 31, seq=1 << 31) == UNS
    assert fwd(T=(1 << 63) - 1, seq=1) == UNS
    assert fwd(T=(1 << 23) + 1, seq=1) == UNS and b"sequences" in L.moe_last_error()
    assert fwd(logits=None) == INV and fwd(idx=None) == INV and fwd(counts=None) == INV and fwd(loss=None) == INV
    assert fwd(tokens=None) == INV and fwd(tokens=ODD) == INV and fwd(logits=ODD) == INV
    assert fwd(nbytes=0) == WS and fwd(ws=None) == INV and fwd(ws=ctypes.c_void_p(4100)) == INV

    def bwd(logits=D, counts=D, tokens=D, T=64, E=8, k=2, seq=64, g=None, d_in=None, d=D):
        return L.moe_balance_loss_bwd(logits, counts, tokens, None, T, E, k, seq, 1.0, 0.0, g, d_in, d, None)

    assert bwd(E=300) == INV and bwd(k=9) == INV and bwd(seq=7) == INV and bwd(logits=None) == INV
    assert bwd(T=1 << 24, seq=1) == UNS
    assert bwd(d=None) == INV and bwd(d=ODD) == INV and bwd(g=ODD) == INV and bwd(d_in=ODD) == INV
    assert bwd(T=0, logits=None) == 0
    st, n = _size(L, _lib.MOE_OP_BALANCE_LOSS, None, 4096, 16384, 128, 0)
    assert st == 0 and n > 0
    assert _size(L, _lib.MOE_OP_BALANCE_LOSS, None, 5, 16384, 128, 0)[0] == INV
    assert _size(L, _lib.MOE_OP_BALANCE_LOSS, None, 0, 16384, 128, 0)[0] == INV
    assert _size(L, _lib.MOE_OP_BALANCE_LOSS, None, 1, 0, 128, 0) == (0, 0)
    assert _size(L, _lib.MOE_OP_BALANCE_LOSS, None, 1, 1, 256, 0) == (0, 0)   # one workgroup


def test_pre_norm(L):
    def fwd(x=D, w=D, dt=1, T=4, H=64, eps=1e-6, y=D, r=None):
        return L.moe_pre_norm(x, w, dt, T, H, eps, y, r, None)

    assert fwd(dt=2) == UNS and fwd(T=-1) == INV and fwd(H=0) == INV and fwd(H=16385) == UNS and fwd(T=1 << 31) == UNS
    assert fwd(eps=0.0) == INV and fwd(eps=float("nan")) == INV and fwd(x=None) == INV and fwd(w=None) == INV
    assert fwd(y=None) == INV and fwd(x=ODD) == INV and fwd(r=ctypes.c_void_p(4098)) == INV
    assert fwd(T=0, x=None) == 0

    def bwd(dy=D, x=D, w=D, r=D, dx_in=None, dt=1, T=4, H=64, dx=D, dw=D, ws=D, n=1 << 20):
        return L.moe_pre_norm_bwd(dy, x, w, r, dx_in, 1.0, dt, T, H, dx, dw, ws, n, None)

    assert bwd(dt=3) == UNS and bwd(dw=None) == INV and bwd(dy=None) == INV and bwd(r=None) == INV and bwd(dx=None) == INV
    assert bwd(dx_in=ODD) == INV and bwd(n=0) == WS and bwd(ws=None) == INV and bwd(ws=ctypes.c_void_p(4112)) == INV


def test_post_norm(L):
    def fwd(y=D, rows=D, k=2, x=D, w=D, kind=0, gate=None, group=1, nw=None, dt=1, T=4, H=64, eps=1e-6, out=D, c=None,
            r=None, yn=None, rn=None):
        return L.moe_post_norm(y, rows, k, x, w, kind, gate, group, 1.0, nw, dt, T, H, eps, out, c, r, yn, rn, None)

    assert fwd(k=0) == INV and fwd(k=17) == UNS and fwd(rows=None) == INV and fwd(T=1 << 30) == UNS
    assert fwd(kind=3, gate=D) == INV and fwd(kind=1) == INV and fwd(kind=2, gate=D, group=0) == INV
    assert fwd(nw=D) == INV and fwd(yn=D) == INV and fwd(eps=0.0) == INV and fwd(out=None) == INV and fwd(x=None) == INV
    assert fwd(rows=ctypes.c_void_p(4098)) == INV and fwd(c=ODD) == INV and fwd(T=0, y=None) == 0

    def bwd(dout=D, c=D, r=D, w=D, kind=0, gate=None, group=1, rows=None, k=1, dt=1, T=4, H=64, dy=D, dw=D, dg=None,
            ws=D, n=1 << 20):
        return L.moe_post_norm_bwd(dout, c, r, w, kind, gate, group, rows, k, dt, T, H, dy, dw, dg, ws, n, None)

    assert bwd(k=2) == INV and bwd(kind=2) == INV and bwd(kind=-1) == INV and bwd(c=None) == INV and bwd(dy=None) == INV
    assert bwd(dw=ODD) == INV and bwd(dg=ODD) == INV and bwd(n=0) == WS and bwd(ws=None) == INV
    d = _lib.MlpDesc(1, 4096, 1, 0, 0, 0, 0)
    # 512 runs of partial column sums, whatever the gate is shared by
    for kind, group in ((0, 0), (1, 0), (2, 4096), (2, 1)):
        st, n = _size(L, _lib.MOE_OP_NORM_BWD, d, 0, 4096, kind, group)
        assert st == 0 and 0 < n <= 2048 * 4096 * 4
    assert _size(L, _lib.MOE_OP_NORM_BWD, d, 0, 0, 0, 0) == (0, 0)
    assert _size(L, _lib.MOE_OP_NORM_BWD, None, 0, 4, 0, 0)[0] == INV
    assert _size(L, _lib.MOE_OP_NORM_BWD, d, 0, 4, 3, 0)[0] == INV
    assert _size(L, _lib.MOE_OP_NORM_BWD, d, 0, 4, 2, 0)[0] == INV


def test_mxfp4(L):
    assert L.mxfp4_quantize(D, 4, 48, D, D, None) == INV and L.mxfp4_quantize(D, -1, 64, D, D, None) == INV
    assert L.mxfp4_quantize(None, 4, 64, D, D, None) == INV and L.mxfp4_quantize(D, 4, 64, ODD, D, None) == INV
    assert L.mxfp4_quantize(ctypes.c_void_p(4104), 4, 64, D, D, None) == INV and L.mxfp4_quantize(None, 0, 64, None, None, None) == 0
    assert L.mxfp4_dequantize(D, D, 4, 40, D, None) == INV and L.mxfp4_dequantize(D, None, 4, 64, D, None) == INV
    assert L.mxfp4_dequantize(D, D, 4, 64, ctypes.c_void_p(4104), None) == INV
    assert L.mxfp4_dequantize(None, None, 4, 0, None, None) == 0
    tab = _lib.ptr_table([4096, 4352, 4608, 4864])[0]
    f = L.moe_pointer_table
    arr = (ctypes.c_void_p * 4)()
    assert f(4096, 256, 4, arr) == 0 and list(arr) == [4096, 4352, 4608, 4864]
    assert f(None, 256, 4, arr) == INV and f(4096, 256, 4, None) == INV and f(4096, 256, -1, arr) == INV and f(4096, 0, 0, None) == 0
    nul = _lib.ptr_table([4096, 4096, None, 4096])[0]
    odd = _lib.ptr_table([4096, 4096, 4100, 4096])[0]
    A, M = _lib.MOE_BF16, _lib.MOE_MXFP4

    def lin(E=4, R=64, K=256, N=256, act=A, x=D, xs=None, w=tab, ws=tab, off=D, y=D, buf=D, n=1 << 20):
        return L.moe_grouped_linear_mxfp4(E, R, K, N, act, x, xs, w, ws, off, y, buf, n, None)

    assert lin(E=0) == INV and lin(E=257) == INV and lin(E=129) == UNS and lin(R=-1) == INV and lin(R=1 << 31) == INV
    assert lin(K=128) == UNS and lin(N=320) == UNS and lin(act=_lib.MOE_MXFP8) == INV and lin(K=1 << 16, N=1 << 16) == UNS
    assert lin(x=None) == INV and lin(y=ODD) == INV and lin(off=None) == INV and lin(w=None) == INV and lin(ws=None) == INV
    assert lin(w=nul) == INV and b"expert 2" in L.moe_last_error()
    assert lin(w=odd) == INV and lin(ws=odd) == INV and lin(act=M) == INV and lin(act=M, xs=ctypes.c_void_p(4100)) == INV
    assert lin(n=16) == WS and lin(buf=None) == INV and lin(buf=ctypes.c_void_p(4112)) == INV and lin(R=0, x=None) == 0
    Desc = _lib.MlpDesc
    assert _size(L, _lib.MOE_OP_LINEAR_MXFP4, Desc(4, 256, 256, M, A, M, 0), 64, 0, 0, 0)[1] >= 64 * (128 + 8)
    assert _size(L, _lib.MOE_OP_LINEAR_MXFP4, Desc(4, 256, 256, M, 0, M, 0), 64, 0, 0, 0)[0] == INV
    assert _size(L, _lib.MOE_OP_LINEAR_MXFP4, None, 64, 0, 0, 0)[0] == INV
    st, n = _size(L, _lib.MOE_OP_MLP_FWD, Desc(8, 512, 256, M, A, A, 0), 64, 0, 0, 0)
    assert st == 0 and n >= 8 * 3 * 512 * 256 // 2 + 64 * (512 + 256) // 2
    assert _size(L, _lib.MOE_OP_MLP_FWD, Desc(8, 512, 256, M, A, A, 1), 64, 0, 0, 0)[0] == UNS     # forward only
    assert _size(L, _lib.MOE_OP_MLP_BWD, Desc(8, 512, 256, M, A, A, 0), 64, 0, 0, 0)[0] == UNS
    assert _size(L, _lib.MOE_OP_MLP_FWD, Desc(129, 512, 256, M, A, A, 0), 64, 0, 0, 0)[0] == UNS
    assert _size(L, _lib.MOE_OP_MLP_FWD, Desc(8, 512, 384, M, A, A, 0), 64, 0, 0, 0)[0] == UNS
    assert _size(L, _lib.MOE_OP_MLP_FWD, Desc(8, 512, 256, M, _lib.MOE_MXFP8, M, 0), 64, 0, 0, 0)[0] == INV
    d = Desc(4, 256, 256, M, M, M, 0)
    fwd = lambda xs=D, s=tab: L.moe_grouped_mlp_fwd(ctypes.byref(d), 64, D, xs, tab, tab, s, tab, D, D, D, None, None, D, 0,
                                                    None)
    assert fwd() == WS and fwd(xs=None) == INV and fwd(xs=ctypes.c_void_p(4100)) == INV and fwd(s=None) == INV and fwd(s=odd) == INV
    assert L.moe_grouped_gate_up_swiglu(4, 64, 256, 256, M, D, D, tab, tab, D, D, D, D, None, None, 0, None) == INV
