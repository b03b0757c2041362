"""What stands around the expert feed-forward in a decoder layer (test infrastructure
only): the router's load-balance loss and the norms before and after the block.

All arithmetic is float64, one sequence or one token at a time.
"""
from __future__ import annotations

import numpy as np

__all__ = ["balance_loss", "balance_loss_backward", "pre_norm", "pre_norm_backward", "post_norm",
           "post_norm_backward", "gate_rows"]

f64 = np.float64


def _counted(logits, mask, s, L):
    """Rows of sequence s that count: not masked out, and not all -infinity."""
    t = np.arange(s * L, (s + 1) * L)
    if mask is not None:
        t = t[np.asarray(mask)[t] != 0]
    return t[~np.all(np.isneginf(logits[t]), axis=1)]


def _softmax_lse(l):
    mx = l.max(axis=1, keepdims=True)
    ex = np.exp(l - mx)
    den = ex.sum(axis=1, keepdims=True)
    return ex / den, (mx + np.log(den))[:, 0]


def balance_loss(logits, topk_idx, balance_coef, z_coef=0.0, seq_len=None, mask=None):
    """loss (total, balance, z), counts [S, E], tokens [S + 1].

    Per sequence with N counted tokens: balance = E sum_e f_e P_e, f_e the expert's share
    of the k N slots, P_e its mean softmax probability; z the mean squared log-sum-exp. The
    loss is the mean over the sequences that have counted tokens."""
    l = np.asarray(logits, f64)
    idx = np.asarray(topk_idx)
    T, E = l.shape
    k = idx.shape[1]
    L = seq_len or max(T, 1)
    S = T // L
    counts = np.zeros((S, E), np.int32)
    tokens = np.zeros(S + 1, np.int32)
    bal, zs = [], []
    for s in range(S):
        t = _counted(l, mask, s, L)
        for e in idx[t].ravel():
            if 0 <= e < E:
                counts[s, e] += 1
        tokens[s] = t.size
        if t.size:
            p, lse = _softmax_lse(l[t])
            bal.append(E * np.sum(counts[s] / (k * t.size) * p.mean(axis=0)))
            zs.append(np.mean(lse ** 2))
    tokens[S] = len(bal)
    b, z = (np.mean(bal), np.mean(zs)) if bal else (0.0, 0.0)
    return np.array([balance_coef * b + z_coef * z, b, z]), counts, tokens


def balance_loss_backward(logits, topk_idx, balance_coef, z_coef=0.0, seq_len=None, mask=None, d_loss=1.0):
    """d loss / d logits times d_loss, the counts held fixed (they are piecewise constant)."""
    l = np.asarray(logits, f64)
    T, E = l.shape
    k = np.asarray(topk_idx).shape[1]
    L = seq_len or max(T, 1)
    _, counts, tokens = balance_loss(l, topk_idx, balance_coef, z_coef, L, mask)
    d = np.zeros((T, E))
    for s in range(T // L):
        t = _counted(l, mask, s, L)
        if not t.size:
            continue
        p, lse = _softmax_lse(l[t])
        f = counts[s] / (k * t.size)
        inner = balance_coef * E * (f - (p * f).sum(axis=1, keepdims=True)) + 2 * z_coef * lse[:, None]
        d[t] = d_loss * p * inner / (tokens[-1] * t.size)
    return d


def pre_norm(x, weight, eps):
    """y = x r weight and r = 1 / sqrt(mean(x^2) + eps), row by row."""
    x = np.asarray(x, f64)
    r = 1.0 / np.sqrt((x * x).mean(axis=1) + eps)
    return x * r[:, None] * np.asarray(weight, f64), r


def _norm_backward(dn, x, r):
    """Gradient of x where n = x r gets the gradient dn: r (dn - n mean(dn n))."""
    n = x * r[:, None]
    return r[:, None] * (dn - n * (dn * n).mean(axis=1, keepdims=True))


def pre_norm_backward(dy, x, weight, r, dx_in=None, dx_in_scale=1.0):
    dy, x, w, r = (np.asarray(a, f64) for a in (dy, x, weight, r))
    dx = _norm_backward(dy * w, x, r)
    if dx_in is not None:
        dx = dx + dx_in_scale * np.asarray(dx_in, f64)
    return dx, (dy * x * r[:, None]).sum(axis=0)


def gate_rows(gate, group, T, H):
    """The gate value of every (token, channel): none, [T], or a row for every `group` tokens."""
    if gate is None:
        return np.ones((T, H))
    g = np.asarray(gate, f64)
    if g.ndim == 1:
        return np.repeat(g[:, None], H, axis=1)
    return g[np.arange(T) // group]


def post_norm(y, x, weight, eps, rows=None, gate=None, group=1, residual_scale=1.0):
    """out, the combined rows c and r. rows [T, k]: each token's rows of y (-1: none)."""
    x, y, w = (np.asarray(a, f64) for a in (x, y, weight))
    T, H = x.shape
    if rows is None:
        c = y
    else:
        c = np.zeros((T, H))
        for t in range(T):
            for r in rows[t]:
                if r >= 0:
                    c[t] += y[r]
    n, r = pre_norm(c, w, eps)
    return residual_scale * x + gate_rows(gate, group, T, H) * n, c, r


def post_norm_backward(dout, c, weight, r, gate=None, group=1):
    """Gradient of c, of the weight, and of the gate (None without one)."""
    dout, c, w, r = (np.asarray(a, f64) for a in (dout, c, weight, r))
    T, H = dout.shape
    g = gate_rows(gate, group, T, H)
    a = dout * c * r[:, None]
    dgate = None
    if gate is not None and np.ndim(gate) == 1:
        dgate = (a * w).sum(axis=1)
    elif gate is not None:
        dgate = np.zeros((np.shape(gate)[0], H))
        for t in range(T):
            dgate[t // group] += a[t] * w
    return _norm_backward(dout * g * w, c, r), (a * g).sum(axis=0), dgate
