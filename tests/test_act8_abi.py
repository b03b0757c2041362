"""Refusals of the operators that hold activations in 8 bits, at the C ABI and in the binding,
before anything is launched (CPU only), and their workspace sizes."""
import ctypes

import pytest
import torch

from grouped_expert_gemm_amd import _lib

INV, UNS, WS = _lib.MOE_ERR_INVALID_ARG, _lib.MOE_ERR_UNSUPPORTED, _lib.MOE_ERR_WORKSPACE
F32, BF16, MXFP8 = _lib.MOE_F32, _lib.MOE_BF16, _lib.MOE_MXFP8
D = ctypes.c_void_p(4096)
E8 = ctypes.c_void_p(4104)    # 8-byte aligned
E4 = ctypes.c_void_p(4100)    # 4-byte aligned
ODD = ctypes.c_void_p(4097)
TAB = (ctypes.c_void_p * 4)(4096, 4352, 4608, 4864)
NUL = (ctypes.c_void_p * 4)(4096, 4352, None, 4864)
BAD = (ctypes.c_void_p * 4)(4096, 4352, 4616, 4864)


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(_lib.LIB_PATH):
        from grouped_expert_gemm_amd import build
        build.build()
    return _lib.lib()


def test_add_norm(L):
    def f(x=D, rows=None, k=1, res=None, w=D, dt=BF16, T=4, H=64, eps=1e-6, s=None, y=None, r=None, c=D, sc=D):
        return L.moe_add_norm_mxfp8(x, rows, k, res, w, dt, T, H, eps, s, y, r, c, sc, None)

    assert f(dt=MXFP8) == UNS and f(T=-1) == INV and f(H=0) == INV and f(H=16416) == UNS and f(H=48) == UNS
    assert f(k=0) == INV and f(k=17, rows=D) == UNS and f(k=2) == INV and b"row_id_map" in L.moe_last_error()
    assert f(k=2, rows=D, T=1 << 30) == UNS and f(T=1 << 31) == UNS
    assert f(eps=0.0) == INV and f(eps=float("nan")) == INV
    assert f(x=None) == INV and f(w=None) == INV and f(c=None) == INV and f(sc=None) == INV
    for name in ("x", "res", "w", "s", "y"):
        assert f(**{name: E8}) == INV, name
    assert f(c=E4) == INV and f(r=ODD) == INV and f(rows=ODD) == INV
    assert f(rows=D, s=D) == INV and b"sum may be x" in L.moe_last_error()
    assert f(T=0, x=None) == 0


def test_dequantize(L):
    def f(c=D, s=D, n=4, cols=64, src=None, rows=4, out=D):
        return L.mxfp8_dequantize(c, s, n, cols, src, rows, out, None)

    assert f(n=-1) == INV and f(cols=-32) == INV and f(rows=-1) == INV and f(cols=40) == INV
    assert f(rows=5) == INV and b"src_row" in L.moe_last_error()
    assert f(rows=1 << 31, src=D) == UNS and f(n=1 << 31, src=D) == UNS and f(cols=1 << 31) == UNS
    assert f(c=None) == INV and f(s=None) == INV and f(out=None) == INV
    assert f(c=E8) == INV and f(out=E8) == INV and f(src=ODD) == INV
    assert f(n=0, rows=0, c=None, s=None, out=None) == 0 and f(cols=0, c=None, s=None, out=None) == 0


def _size(L, desc, R, op=_lib.MOE_OP_MLP_BWD_CKPT8):
    n = ctypes.c_size_t()
    st = L.moe_workspace_size(op, ctypes.byref(desc) if desc else None, R, 0, 0, 0, ctypes.byref(n))
    return st, n.value


def _bad_descs(backward):
    d = _lib.MlpDesc
    ok_act = (BF16, MXFP8) if backward else (BF16,)
    yield d(0, 256, 256, BF16, BF16, BF16, 0), INV
    yield d(257, 256, 256, BF16, BF16, BF16, 0), INV
    yield d(4, 0, 256, BF16, BF16, BF16, 0), INV
    yield d(4, 128, 256, BF16, BF16, BF16, 0), UNS
    yield d(4, 256, 128, BF16, BF16, BF16, 0), UNS
    yield d(4, 1 << 16, 1 << 15, BF16, BF16, BF16, 0), UNS
    for c in (F32, MXFP8, _lib.MOE_FP8, _lib.MOE_MXFP4):
        yield d(4, 256, 256, c, BF16, BF16, 0), UNS
        yield d(4, 256, 256, BF16, BF16, c, 0), UNS
        if c not in ok_act:
            yield d(4, 256, 256, BF16, c, BF16, 0), UNS


def test_forward(L):
    good = _lib.MlpDesc(4, 256, 512, BF16, BF16, BF16, 1)   # save_for_bwd plays no part

    def f(d=good, R=8, x=D, w1=TAB, w2=TAB, off=D, p=D, y=D, zc=D, zs=D, ws=D, n=1 << 40):
        return L.moe_grouped_mlp_fwd_ckpt8(ctypes.byref(d) if d else None, R, x, w1, w2, off, p, y, zc, zs, ws, n, None)

    assert f(d=None) == INV and f(R=-1) == INV and f(R=1 << 31) == INV
    for d, want in _bad_descs(False):
        assert f(d=d) == want, tuple(getattr(d, n) for n, _ in d._fields_)
    for name in ("x", "off", "p", "y", "zc", "zs"):
        assert f(**{name: None}) == INV and f(**{name: ODD}) == INV, name
    for name in ("x", "y", "zc"):
        assert f(**{name: E8}) == INV, name
    for name in ("w1", "w2"):
        assert f(**{name: None}) == INV and f(**{name: NUL}) == INV and b"expert 2" in L.moe_last_error()
        assert f(**{name: BAD}) == INV, name
    st, need = _size(L, _lib.MlpDesc(4, 256, 512, BF16, BF16, BF16, 0), 8, _lib.MOE_OP_MLP_FWD)
    assert st == 0 and f(n=need - 1) == WS and f(n=need, ws=None) == INV and f(n=need, ws=ctypes.c_void_p(4224)) == INV
    assert f(R=0, x=None) == 0


def test_backward(L):
    good = _lib.MlpDesc(4, 512, 256, BF16, MXFP8, BF16, 0)
    plain = _lib.MlpDesc(4, 512, 256, BF16, BF16, BF16, 0)

    def f(d=good, R=8, dy=D, x=D, xs=D, T=4, src=D, zc=D, zs=D, p=D, w1=TAB, w2=TAB, off=D, dx=D, d1=TAB, d2=TAB, dp=D,
          ws=D, n=1 << 40):
        return L.moe_grouped_mlp_bwd_ckpt8(ctypes.byref(d) if d else None, R, dy, x, xs, T, src, zc, zs, p, w1, w2, off, dx,
                                           d1, d2, dp, ws, n, None)

    assert f(d=None) == INV and f(R=-1) == INV and f(R=1 << 31) == INV
    for d, want in _bad_descs(True):
        assert f(d=d) == want and _size(L, d, 8)[0] == want, tuple(getattr(d, n) for n, _ in d._fields_)
    for name in ("dy", "x", "xs", "zc", "zs", "p", "off", "dx", "dp"):
        assert f(**{name: None}) == INV, name
    for name in ("dy", "x", "zc", "dx"):
        assert f(**{name: E8}) == INV, name
    for name in ("src", "p", "off", "dp"):
        assert f(**{name: ODD}) == INV, name
    assert f(zs=E4) == INV and f(T=-1) == INV and f(T=1 << 31) == INV
    assert f(src=None) == INV and b"src_token" in L.moe_last_error()
    assert f(d=plain, xs=None) == INV and f(d=plain, src=None) == INV     # what belongs to codes alone
    for name in ("w1", "w2", "d1", "d2"):
        assert f(**{name: None}) == INV and f(**{name: NUL}) == INV and f(**{name: BAD}) == INV, name
    st, need = _size(L, good, 8)
    assert st == 0 and f(n=need - 1) == WS and f(n=need, ws=None) == INV and f(n=need, ws=ctypes.c_void_p(4224)) == INV
    assert _size(L, None, 8)[0] == INV and _size(L, good, -1)[0] == INV and _size(L, good, 1 << 31)[0] == INV
    # dZ, and the wider of h and x, in bf16
    big = 100000
    assert _size(L, good, big)[1] >= 2 * big * (512 + 512) and _size(L, plain, big)[1] < _size(L, good, big)[1]


def test_binding_refuses_cpu_tensors():
    import grouped_expert_gemm_amd as moe
    x, w = torch.zeros(4, 64), torch.ones(64)
    with pytest.raises(ValueError, match="moe_add_norm_mxfp8"):
        moe.moe_add_norm_mxfp8(x, w)
    c, s = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="mxfp8_dequantize"):
        moe.mxfp8_dequantize(c, s)
    with pytest.raises(ValueError, match="moe_grouped_mlp_fwd_ckpt8"):
        moe.moe_grouped_mlp_fwd_ckpt8(x.bfloat16(), w, w, w, w)
    with pytest.raises(ValueError, match="moe_grouped_mlp_bwd_ckpt8"):
        moe.moe_grouped_mlp_bwd_ckpt8(x.bfloat16(), c, c, s, w, w, w, w)
