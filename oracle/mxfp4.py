"""MXFP4: block quantisation, products and the grouped MLP forward, as a plain CPU
reference (test infrastructure only).

* elements are OCP FP4 E2M1: sign in bit 3, magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 for the
  codes 0..7; two codes a byte, the even element in the low nibble;
* the scale is an E8M0 power of two 2^s stored as s + 127, one per 32 contiguous values
  along the GEMM's reduction axis; s is the smallest integer with max|block| <= 6 * 2^s,
  clamped to [-127, 127], -127 for an all-zero block; byte 255 and codes 0 for a block that
  holds an infinity or a NaN (its values are NaN);
* a code is the nearest magnitude to |x| / 2^s, ties to the even code, with x's sign bit.
"""
from __future__ import annotations

import numpy as np

__all__ = ["E2M1_VALUES", "mxfp4_encode", "mxfp4_pack", "mxfp4_unpack", "mxfp4_quantize", "mxfp4_dequantize",
           "mxfp4_qdq", "mxfp4_mlp_forward"]

f64 = np.float64
E2M1_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _scale_exponent(amax):
    """Smallest s with amax <= 6 * 2^s, by exact comparison around the logarithm."""
    with np.errstate(divide="ignore"):
        s = np.where(amax > 0, np.floor(np.log2(np.where(amax > 0, amax, 1.0))) - 4, -127).astype(np.int64)
    for _ in range(4):
        s = np.where((amax > 0) & (amax > np.ldexp(6.0, s)), s + 1, s)
    return np.clip(s, -127, 127)


def mxfp4_encode(x):
    """x [..., cols] -> (codes 0..15 [..., cols], scale bytes [..., cols/32])."""
    x = np.asarray(x, f64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    bad = ~np.all(np.isfinite(b), axis=-1)
    amax = np.max(np.abs(np.where(np.isfinite(b), b, 0)), axis=-1)
    s = _scale_exponent(amax)
    a = np.abs(np.where(bad[..., None], 0.0, b)) / np.ldexp(1.0, s)[..., None]
    # nearest codebook entry; of two equally near ones the even code
    dist = np.abs(a[..., None] - E2M1_VALUES)
    best = dist.min(axis=-1, keepdims=True)
    code = np.argmax((dist == best) * np.where(np.arange(8) % 2 == 0, 2, 1), axis=-1)
    code = code + 8 * (np.signbit(b) & ~bad[..., None])
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 255, s + 127).astype(np.uint8)


def mxfp4_pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def mxfp4_unpack(packed):
    out = np.empty((*packed.shape[:-1], 2 * packed.shape[-1]), np.uint8)
    out[..., 0::2], out[..., 1::2] = packed & 15, packed >> 4
    return out


def mxfp4_quantize(x):
    codes, scales = mxfp4_encode(x)
    return mxfp4_pack(codes), scales


def mxfp4_dequantize(packed, scales):
    c = mxfp4_unpack(np.asarray(packed))
    v = np.where(c & 8, -1.0, 1.0) * E2M1_VALUES[c & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, np.asarray(scales).astype(np.int64) - 127))
    return (v.reshape(*scales.shape, 32) * s[..., None]).reshape(v.shape)


def mxfp4_qdq(x):
    return mxfp4_dequantize(*mxfp4_quantize(x))


def mxfp4_mlp_forward(x_perm, w1, w2, offsets, prob, h_quantise=mxfp4_qdq):
    """y and the float64 h of the grouped MLP on MXFP4 operand values: x_perm quantised along
    its rows, w1 [E, 2I, H] and w2 [E, H, I] given as the values of their codes, h quantised."""
    x = mxfp4_qdq(x_perm)
    p = np.asarray(prob, f64)
    I = w1.shape[1] // 2
    y = np.zeros((x.shape[0], w2.shape[1]))
    hs = np.zeros((x.shape[0], I))
    for e in range(w1.shape[0]):
        r = slice(int(offsets[e]), int(offsets[e + 1]))
        z = x[r] @ w1[e].T
        h = z[:, :I] / (1 + np.exp(-z[:, :I])) * z[:, I:] * p[r, None]
        hs[r] = h
        if h.shape[0]:
            y[r] = h_quantise(h) @ w2[e].T
    return y, hs
