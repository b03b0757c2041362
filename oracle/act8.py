"""Activations held in 8 bits between the forward and the backward (test infrastructure only):
the norm that adds the residual, and the grouped MLP's backward from its kept gate_up output.

All arithmetic is float64.
"""
from __future__ import annotations

import numpy as np

__all__ = ["add_rows", "mxfp8_bounds", "grouped_mlp_backward_from_z"]

from .mxfp8 import e4m3_decode, e4m3_encode, e8m0_scale_exponent

f64 = np.float64


def add_rows(x, residual=None, rows=None):
    """residual[t] + sum_j x[rows[t, j]] (entries out of range add nothing), or residual + x."""
    x = np.asarray(x, f64)
    if rows is None:
        s = x.copy()
    else:
        s = np.zeros((len(rows), x.shape[1]), f64)
        for t, js in enumerate(rows):
            for j in js:
                if 0 <= j < len(x):
                    s[t] += x[j]
    return s if residual is None else s + np.asarray(residual, f64)


def mxfp8_bounds(v, err, scales):
    """The MXFP8 values that a block's elements may be read back as when each was known only to
    lie within v +- err before it was rounded: (lo, hi) for the given scale bytes, and whether
    each scale byte is that of a possible block maximum. Rounding is monotone, so an
    element's result lies between the results of its interval's ends."""
    v, err = np.asarray(v, f64), np.asarray(err, f64)
    rows, cols = v.shape
    blk = lambda a: a.reshape(rows, cols // 32, 32)
    s = np.asarray(scales, np.int64) - 127
    top_lo = np.maximum(np.abs(blk(v)) - blk(err), 0).max(axis=2)
    top_hi = (np.abs(blk(v)) + blk(err)).max(axis=2)
    ok = (e8m0_scale_exponent(top_lo) <= s) & (s <= e8m0_scale_exponent(top_hi))
    step = np.exp2(s.astype(f64))[:, :, None]
    q = lambda a: (e4m3_decode(e4m3_encode(blk(a) / step)) * step).reshape(rows, cols)
    return q(v - err), q(v + err), ok


def grouped_mlp_backward_from_z(dy_perm, x_perm, z, w_gate_up, w_down, offsets, prob_perm):
    """Gradients of y = (silu(G) U p) W2^T, (G, U) = the given z, and of z = x W1^T, per expert:
    dict dx_perm, dw_gate_up, dw_down, dprob_perm, and the intermediate dz [R, 2I] and h [R, I].
    Rows outside every expert keep zeros."""
    dy, x, z = (np.asarray(a, f64) for a in (dy_perm, x_perm, z))
    p, off = np.asarray(prob_perm, f64), np.asarray(offsets, np.int64)
    E, twoI, H = np.shape(w_gate_up)
    I, R = twoI // 2, dy.shape[0]
    out = dict(dx_perm=np.zeros((R, H)), dw_gate_up=np.zeros((E, twoI, H)), dw_down=np.zeros((E, H, I)),
               dprob_perm=np.zeros(R), dz=np.zeros((R, twoI)), h=np.zeros((R, I)))
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if r.start == r.stop:
            continue
        w1, w2 = np.asarray(w_gate_up[e], f64), np.asarray(w_down[e], f64)
        g, u, pe = z[r, :I], z[r, I:], p[r, None]
        sig = np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))
        act = g * sig * u
        dh = dy[r] @ w2
        out["h"][r] = act * pe
        out["dprob_perm"][r] = (dh * act).sum(1)
        # d silu / dg = sig + g sig (1 - sig)
        out["dz"][r] = np.concatenate([dh * pe * u * (sig + g * sig * (1 - sig)), dh * pe * g * sig], 1)
        out["dx_perm"][r] = out["dz"][r] @ w1
        out["dw_gate_up"][e] = out["dz"][r].T @ x[r]
        out["dw_down"][e] = dy[r].T @ out["h"][r]
    return out
