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
    def fwd(logits=D, idx=D, T=64, E=8, k=2, seq=64, counts=D, tokens=D, loss=D, ws=D, nbytes=1 << 20):
        return L.moe_balance_loss(logits, idx, None, T, E, k, seq, 1.0, 0.0, counts, tokens, loss, ws, nbytes, None)

    assert fwd(T=-1) == INV and fwd(E=0) == INV and fwd(E=257) == INV and fwd(k=0) == INV and fwd(k=9) == INV
    assert fwd(seq=0) == INV and fwd(seq=63) == INV and b"seq_len" in L.moe_last_error()
    assert fwd(T=1 << 31, seq=1 << 31) == UNS
    assert fwd(T=(1 << 63) - 1, seq=1) == UNS
    assert fwd(logits=None) == INV and fwd(idx=None) == INV and fwd(counts=None) == INV and fwd(loss=None) == INV
    assert fwd(tokens=None) == INV and fwd(tokens=ODD) == INV and fwd(logits=ODD) == INV
    assert fwd(nbytes=0) == WS and fwd(ws=None) == INV and fwd(ws=ctypes.c_void_p(4100)) == INV

    def bwd(logits=D, counts=D, tokens=D, T=64, E=8, k=2, seq=64, g=None, d_in=None, d=D):
        return L.moe_balance_loss_bwd(logits, counts, tokens, None, T, E, k, seq, 1.0, 0.0, g, d_in, d, None)

    assert bwd(E=300) == INV and bwd(k=9) == INV and bwd(seq=7) == INV and bwd(logits=None) == INV
    assert bwd(d=None) == INV and bwd(d=ODD) == INV and bwd(g=ODD) == INV and bwd(d_in=ODD) == INV
    assert bwd(T=0, logits=None) == 0
    st, n = _size(L, _lib.MOE_OP_BALANCE_LOSS, None, 4096, 16384, 128, 0)
    assert st == 0 and n > 0
    assert _size(L, _lib.MOE_OP_BALANCE_LOSS, None, 5, 16384, 128, 0)[0] == INV
    assert _size(L, _lib.MOE_OP_BALANCE_LOSS, None, 0, 16384, 128, 0)[0] == INV
    assert _size(L, _lib.MOE_OP_BALANCE_LOSS, None, 1, 0, 128, 0)[0] == 0


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
