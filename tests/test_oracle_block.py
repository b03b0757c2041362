"""The oracle of the balance loss and the norms around the block: closed forms, invariants
and finite differences of its own forwards (CPU)."""
import numpy as np
import pytest

import oracle


def _routed(rng, T, E, k, spread=1.0):
    logits = spread * rng.standard_normal((T, E))
    return logits, np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)


def test_balance_is_one_for_even_loads_and_probabilities():
    E, k = 8, 2
    idx = np.array([[(2 * t) % E, (2 * t + 1) % E] for t in range(16)], np.int32)
    loss, counts, tokens = oracle.balance_loss(np.zeros((16, E)), idx, 0.5, 0.25)
    assert np.all(counts == 4) and tokens.tolist() == [16, 1]
    assert loss[1] == pytest.approx(1.0) and loss[2] == pytest.approx(np.log(E) ** 2)
    assert loss[0] == pytest.approx(0.5 + 0.25 * np.log(E) ** 2)


def test_balance_of_one_expert_taking_all_is_E_times_its_probability():
    logits = np.tile([3.0, 0.0, 0.0, 0.0], (5, 1))
    p0 = np.exp(3) / (np.exp(3) + 3)
    loss, counts, _ = oracle.balance_loss(logits, np.zeros((5, 1), np.int32), 1.0)
    assert counts[0].tolist() == [5, 0, 0, 0] and loss[0] == pytest.approx(4 * p0)


@pytest.mark.parametrize("seq_len,masked", [(12, False), (4, True), (3, True)])
def test_balance_gradient_is_that_of_differences(seq_len, masked):
    rng = np.random.default_rng(3)
    T, E, k = 12, 5, 2
    logits, idx = _routed(rng, T, E, k)
    mask = None
    if masked:
        mask = rng.integers(0, 2, T).astype(np.uint8)
        mask[:seq_len] = 0          # a sequence that is all padding
    d = oracle.balance_loss_backward(logits, idx, 0.7, 0.3, seq_len, mask, d_loss=1.5)
    for t in range(T):
        for e in range(E):
            hi, lo = logits.copy(), logits.copy()
            hi[t, e] += 1e-5
            lo[t, e] -= 1e-5
            f = [1.5 * oracle.balance_loss(l, idx, 0.7, 0.3, seq_len, mask)[0][0] for l in (hi, lo)]
            assert (f[0] - f[1]) / 2e-5 == pytest.approx(d[t, e], abs=1e-8)
    assert masked is False or np.all(d[mask == 0] == 0)


def test_rows_without_a_finite_logit_do_not_count():
    logits = np.array([[0.0, 1.0], [-np.inf, -np.inf], [-np.inf, 2.0]])
    loss, counts, tokens = oracle.balance_loss(logits, np.array([[1], [0], [1]], np.int32), 1.0)
    assert tokens.tolist() == [2, 1] and counts.tolist() == [[0, 2]] and np.all(np.isfinite(loss))


@pytest.mark.parametrize("gate", ["none", "token", "channel"])
def test_norm_gradients_are_those_of_differences(gate):
    rng = np.random.default_rng(5)
    T, H, k, eps, group = 5, 6, 2, 1e-3, 2
    y, x, w = rng.standard_normal((T * k, H)), rng.standard_normal((T, H)), rng.standard_normal(H)
    rows = rng.permutation(T * k).reshape(T, k)
    rows[3, 1] = -1
    g = {"none": None, "token": rng.standard_normal(T), "channel": rng.standard_normal((3, H))}[gate]
    dout = rng.standard_normal((T, H))

    def f(y_, w_, g_):
        return float((dout * oracle.post_norm(y_, x, w_, eps, rows, g_, group, 0.5)[0]).sum())

    _, c, r = oracle.post_norm(y, x, w, eps, rows, g, group, 0.5)
    dc, dw, dg = oracle.post_norm_backward(dout, c, w, r, g, group)

    def diff(a, i, call):
        hi, lo = a.copy(), a.copy()
        hi[i] += 1e-6
        lo[i] -= 1e-6
        return (call(hi) - call(lo)) / 2e-6

    for t in range(T):
        for row in rows[t]:
            if row >= 0:
                assert diff(y, (row, 3), lambda v: f(v, w, g)) == pytest.approx(dc[t, 3], abs=1e-6)
    for h in range(H):
        assert diff(w, h, lambda v: f(y, v, g)) == pytest.approx(dw[h], abs=1e-6)
    if g is not None:
        for i in np.ndindex(*g.shape):
            assert diff(g, i, lambda v: f(y, w, v)) == pytest.approx(dg[i], abs=1e-6)


def test_pre_norm_rows_have_unit_mean_square_and_their_gradient():
    rng = np.random.default_rng(6)
    x, w, dy, dx_in = rng.standard_normal((4, 7)), rng.standard_normal(7), rng.standard_normal((4, 7)), rng.standard_normal((4, 7))
    y, r = oracle.pre_norm(x, np.ones(7), 1e-12)
    assert np.allclose((y * y).mean(axis=1), 1.0)
    _, r = oracle.pre_norm(x, w, 1e-3)
    dx, dw = oracle.pre_norm_backward(dy, x, w, r, dx_in, 2.0)
    for i in np.ndindex(4, 7):
        hi, lo = x.copy(), x.copy()
        hi[i] += 1e-6
        lo[i] -= 1e-6
        num = (dy * (oracle.pre_norm(hi, w, 1e-3)[0] - oracle.pre_norm(lo, w, 1e-3)[0])).sum() / 2e-6
        assert num + 2 * dx_in[i] == pytest.approx(dx[i], abs=1e-6)
    assert np.allclose(dw, (dy * x * r[:, None]).sum(axis=0))
