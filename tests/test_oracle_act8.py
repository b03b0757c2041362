"""Pins of the oracle's 8-bit activation parts (CPU only)."""
import numpy as np
import torch

import oracle


def test_add_rows_by_hand():
    x = np.arange(12.0).reshape(4, 3)
    rows = np.array([[3, 0], [-1, 2], [-1, -1], [4, 1]])   # 4 is out of range
    want = np.array([[9, 11, 13], [6, 7, 8], [0, 0, 0], [3, 4, 5]], float)
    assert np.array_equal(oracle.add_rows(x, None, rows), want)
    assert np.array_equal(oracle.add_rows(x, np.ones((4, 3)), rows), want + 1)
    assert np.array_equal(oracle.add_rows(x, np.ones((4, 3))), x + 1)


def test_bounds_hold_every_value_of_the_interval():
    g = np.random.default_rng(0)
    v = g.standard_normal((40, 64)) * np.exp2(g.integers(-20, 20, (40, 1)))
    err = np.abs(v) * 2.0 ** -6
    for _ in range(20):
        w = v + err * g.uniform(-1, 1, v.shape)
        codes, scales = oracle.mxfp8_quantize(w)
        lo, hi, ok = oracle.mxfp8_bounds(v, err, scales)
        got = oracle.mxfp8_dequantize(codes, scales)
        assert ok.all() and (lo <= got).all() and (got <= hi).all()
    # a value off by a whole E4M3 step, or a scale off by one, falls outside
    codes, scales = oracle.mxfp8_quantize(v)
    lo, hi, _ = oracle.mxfp8_bounds(v, np.abs(v) * 1e-6, scales)
    moved = oracle.mxfp8_dequantize(codes ^ 2, scales)
    assert not ((moved >= lo) & (moved <= hi)).any()        # (a code that became NaN lies outside as well)
    assert not oracle.mxfp8_bounds(v, np.abs(v) * 1e-6, scales + 1)[2].any()


def _case(seed=1):
    g = np.random.default_rng(seed)
    E, H, I, R = 3, 8, 6, 11
    off = np.array([0, 4, 4, 9])                            # an idle expert, two rows behind the last
    w1, w2 = g.standard_normal((E, 2 * I, H)), g.standard_normal((E, H, I))
    x, dy, p = g.standard_normal((R, H)), g.standard_normal((R, H)), g.uniform(0.1, 1, R)
    return E, H, I, R, off, w1, w2, x, dy, p


def test_backward_from_z_is_the_backward():
    E, H, I, R, off, w1, w2, x, dy, p = _case()
    z = np.zeros((R, 2 * I))
    for e in range(E):
        z[off[e]:off[e + 1]] = x[off[e]:off[e + 1]] @ w1[e].T
    got = oracle.grouped_mlp_backward_from_z(dy, x, z, w1, w2, off, p)
    want = oracle.grouped_mlp_backward(dy, x, w1, w2, off, p)
    for k in want:
        assert np.allclose(got[k], want[k], rtol=1e-12, atol=1e-13), k
    assert not got["dw_gate_up"][1].any() and not got["dx_perm"][9:].any()


def test_backward_from_z_against_differences_and_autograd():
    """z given apart from x: dz, dprob and dW2 are gradients of the output alone."""
    E, H, I, R, off, w1, w2, x, dy, p = _case(2)
    z = np.random.default_rng(3).standard_normal((R, 2 * I))
    got = oracle.grouped_mlp_backward_from_z(dy, x, z, w1, w2, off, p)

    def loss(z, p, w2):
        total = 0.0
        for e in range(E):
            r = slice(off[e], off[e + 1])
            h = z[r, :I] / (1 + np.exp(-z[r, :I])) * z[r, I:] * p[r, None]
            total += (dy[r] * (h @ w2[e].T)).sum()
        return total

    g = np.random.default_rng(4)
    for _ in range(10):
        d = [g.standard_normal(a.shape) for a in (z, p, w2)]
        t = 1e-5
        num = (loss(z + t * d[0], p + t * d[1], w2 + t * d[2]) - loss(z - t * d[0], p - t * d[1], w2 - t * d[2])) / (2 * t)
        want = (got["dz"] * d[0]).sum() + (got["dprob_perm"] * d[1]).sum() + (got["dw_down"] * d[2]).sum()
        assert abs(num - want) <= 1e-7 * (1 + abs(want))     # t^2 of a third derivative of order 10, and 1e-16 / t
    # dx and dW1 are those of z = x W1^T with that dz
    tx, tw = (torch.tensor(a, dtype=torch.float64, requires_grad=True) for a in (x, w1))
    s = sum((torch.tensor(got["dz"][off[e]:off[e + 1]]) * (tx[off[e]:off[e + 1]] @ tw[e].T)).sum() for e in range(E))
    s.backward()
    assert np.allclose(tx.grad.numpy(), got["dx_perm"], atol=1e-12) and np.allclose(tw.grad.numpy(), got["dw_gate_up"], atol=1e-12)
