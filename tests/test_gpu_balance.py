"""GPU parity of the load-balance loss and its gradient against the float64 oracle.

Tolerances, from the kernels' float32 arithmetic (u = 2^-24, half a step): a probability is
off by at most (|l - max| + 16) u relative (the rounded difference, exp, the row's sum, the
reciprocal, two products); sums of T probabilities by another 64 u of their absolute sum (the
runs are at most 256 tokens long a lane, in practice far less, and errors of a run average;
the bound taken is 64 u); a gradient multiplies a handful of such factors. Counts are exact."""
import ctypes

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_expert_gemm_amd as g
    g.lib()
    return g


def _inputs(seed, T, E, k, spread=1.0):
    rng = np.random.default_rng(seed)
    logits = (spread * rng.standard_normal((T, E)) + 0.5 * rng.standard_normal((1, E))).astype(np.float32)
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    return rng, logits, np.ascontiguousarray(idx)


def _cuda(a):
    return None if a is None else torch.from_numpy(a).cuda()


def _check(moe, logits, idx, a, b, L, mask, g, d_in, label):
    T, E = logits.shape
    k = idx.shape[1]
    print(f"balance {label}: T={T} E={E} k={k} seq_len={L}", flush=True)
    ref, counts, tokens = oracle.balance_loss(logits, idx, a, b, L, mask)
    d_ref = oracle.balance_loss_backward(logits, idx, a, b, L, mask, 1.0 if g is None else float(g[0]))
    if d_in is not None:
        d_ref = d_ref + d_in
    l, m = _cuda(logits), _cuda(mask)
    loss, c, n = moe.moe_balance_loss(l, _cuda(idx), a, b, seq_len=L, mask=m)
    d = moe.moe_balance_loss_bwd(l, c, n, k, a, b, seq_len=L, mask=m, d_loss=_cuda(g), d_logits_in=_cuda(d_in))
    again = moe.moe_balance_loss(l, _cuda(idx), a, b, seq_len=L, mask=m)
    torch.cuda.synchronize()
    assert np.array_equal(c.cpu().numpy(), counts) and np.array_equal(n.cpu().numpy(), tokens)
    for p, q in zip((loss, c, n), again):
        assert torch.equal(p.view(torch.int32), q.view(torch.int32))
    live = np.isfinite(logits)
    wide = float(np.where(live, np.abs(np.where(live, logits, 0)), 0).max()) * 2 + 16
    tol = (wide + 64) * U * (abs(ref[0]) + 2 * abs(a) + abs(b) * ref[2] + np.abs(ref))
    assert np.all(np.abs(loss.cpu().numpy() - ref) <= tol), (loss.cpu().numpy(), ref)
    # each gradient: |g| / (S' N) p (|a| E max f + |a| + 2 |b| |lse|), relative to that
    S = max(1, T // max(L, 1))
    seqs = max(1, int(tokens[-1]))
    tol = np.zeros((T, E))
    for s in range(S):
        if tokens[s]:
            rows = slice(s * L, (s + 1) * L)
            x = np.where(np.isfinite(logits[rows]), logits[rows], -np.inf).astype(np.float64)
            with np.errstate(invalid="ignore", divide="ignore"):
                mx = x.max(axis=1, keepdims=True)
                p = np.exp(x - mx)
                den = p.sum(axis=1, keepdims=True)
                lse = np.abs(mx + np.log(den))
                p = np.nan_to_num(p / den)
            big = abs(a) * (E * counts[s].max() / (k * tokens[s]) + 1) + 2 * abs(b) * np.nan_to_num(lse, posinf=0, neginf=0)
            tol[rows] = (wide + 16) * U * 2 * p * big / (seqs * tokens[s]) * (1.0 if g is None else abs(float(g[0])))
    tol += 2 * U * np.abs(d_ref) + 1e-44
    err = np.abs(d.cpu().numpy() - d_ref)
    assert np.all(err <= tol), (float((err / tol).max()), np.unravel_index((err / tol).argmax(), err.shape))


# sizes at the kernel's borders: one lane a token, part-filled and 64-lane groups, rows that
# are not a multiple of 16 bytes, one token, one more than a workgroup's share
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (3, 2, 2), (7, 5, 3), (129, 8, 2), (1025, 4, 4), (300, 64, 6),
                                   (517, 100, 8), (2049, 128, 8), (777, 255, 16), (64, 37, 1), (5000, 256, 16)])
def test_against_oracle(moe, T, E, k):
    rng, logits, idx = _inputs(T * 1000 + E, T, E, k)
    _check(moe, logits, idx, 0.01, 0.001, T, None, None, None, "plain")
    g = np.array([-1.75], np.float32)
    d_in = (1e-4 * rng.standard_normal((T, E))).astype(np.float32)
    mask = rng.integers(0, 2, T).astype(np.uint8)
    _check(moe, logits, idx, 1.0, 0.0, T, mask, g, d_in, "masked")


@pytest.mark.parametrize("S,L", [(5, 1), (3, 100), (2, 1500), (700, 3)])
def test_sequences(moe, S, L):
    E, k = 24, 3
    rng, logits, idx = _inputs(S * 7 + L, S * L, E, k)
    mask = (np.arange(L)[None] < rng.integers(0, L + 1, (S, 1))).astype(np.uint8).ravel()
    mask[:L] = 0  # a sequence of padding alone
    _check(moe, logits, idx, 0.5, 0.25, L, mask, np.array([2.0], np.float32), None, "sequences")


def test_nothing_counted_and_no_tokens(moe):
    _, logits, idx = _inputs(1, 40, 6, 2)
    mask = np.zeros(40, np.uint8)
    logits[3] = np.nan          # never read
    d_in = np.full((40, 6), 0.5, np.float32)
    loss, c, n = moe.moe_balance_loss(_cuda(logits), _cuda(idx), 1.0, 1.0, seq_len=10, mask=_cuda(mask))
    d = moe.moe_balance_loss_bwd(_cuda(logits), c, n, 2, 1.0, 1.0, seq_len=10, mask=_cuda(mask), d_logits_in=_cuda(d_in))
    assert loss.tolist() == [0, 0, 0] and int(c.abs().sum()) == 0 and n.tolist() == [0] * 5
    assert torch.all(d == 0.5)
    loss, c, n = moe.moe_balance_loss(torch.empty((0, 6), device="cuda"), torch.empty((0, 2), dtype=torch.int32, device="cuda"), 1.0)
    assert loss.tolist() == [0, 0, 0] and c.shape == (0, 6) and n.tolist() == [0]
    assert moe.moe_balance_loss_bwd(torch.empty((0, 6), device="cuda"), c, n, 2, 1.0).shape == (0, 6)


def test_infinities_masked_experts_and_nan(moe):
    """Logits of -infinity (an expert that is closed), a row of nothing else, the type's lowest
    value, and a masked row full of NaN; then a NaN that counts, which has to show."""
    _, logits, idx = _inputs(2, 50, 12, 4)
    logits[:, 3] = -np.inf
    logits[7] = -np.inf
    logits[9, :] = np.finfo(np.float32).min
    logits[11, 5] = np.finfo(np.float32).min
    mask = np.ones(50, np.uint8)
    mask[20] = 0
    bad = logits.copy()
    bad[20] = np.nan
    l = _cuda(bad)
    loss, c, n = moe.moe_balance_loss(l, _cuda(idx), 1.0, 0.0, mask=_cuda(mask))
    ref, counts, tokens = oracle.balance_loss(logits, idx, 1.0, 0.0, None, mask)
    assert np.array_equal(c.cpu().numpy(), counts) and n.tolist() == tokens.tolist() == [48, 1]
    assert abs(float(loss[0]) - ref[0]) <= 128 * U * (abs(ref[0]) + 2)
    d = moe.moe_balance_loss_bwd(l, c, n, 4, 1.0, 0.0, mask=_cuda(mask)).cpu().numpy()
    d_ref = oracle.balance_loss_backward(logits, idx, 1.0, 0.0, None, mask)
    # (row 9 holds twelve equal finite logits, the closed expert's among them: p = 1/12 each)
    closed = np.isneginf(logits[:, 3])
    assert np.all(np.isfinite(d)) and np.all(d[[7, 20]] == 0) and np.all(d[closed, 3] == 0)
    assert np.abs(d - d_ref).max() <= 256 * U * np.abs(d_ref).max()
    bad[30, 2] = np.nan
    loss, _, _ = moe.moe_balance_loss(_cuda(bad), _cuda(idx), 1.0, 0.0, mask=_cuda(mask))
    assert torch.isnan(loss[0])


def test_dropped_and_repeated_ids(moe):
    logits = np.zeros((4, 4), np.float32)
    idx = np.array([[0, 0], [-1, 1], [9, 3], [2, 2 ** 30]], np.int32)
    _, c, n = moe.moe_balance_loss(_cuda(logits), _cuda(idx), 1.0)
    assert c.tolist() == [[2, 1, 1, 1]] and n.tolist() == [4, 1]


def test_gradient_in_place_unaligned_rows_and_another_stream(moe):
    """d_logits_in overwritten in place; rows that start 4 bytes past a 16-byte border (the
    one-value loads); work queued on a side stream."""
    T, E, k = 333, 32, 4
    rng, logits, idx = _inputs(11, T, E, k)
    d_in = rng.standard_normal((T, E)).astype(np.float32)
    store = torch.empty(T * E + 1, device="cuda")
    l2 = store[1:].view(T, E)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        l2.copy_(_cuda(logits))
        a, c, n = moe.moe_balance_loss(l2, _cuda(idx), 1.0, 0.1)
        d = _cuda(d_in)
        out = moe.moe_balance_loss_bwd(l2, c, n, k, 1.0, 0.1, d_logits_in=d, d_logits=d)
    s.synchronize()
    assert out.data_ptr() == d.data_ptr()
    ref = oracle.balance_loss_backward(logits, idx, 1.0, 0.1) + d_in
    assert np.abs(out.cpu().numpy() - ref).max() <= 64 * U * np.abs(ref).max()


def test_refusals(moe):
    l = torch.zeros((8, 4), device="cuda")
    i = torch.zeros((8, 2), dtype=torch.int32, device="cuda")
    for bad in (lambda: moe.moe_balance_loss(l.cpu(), i, 1.0), lambda: moe.moe_balance_loss(l.t(), i, 1.0),
                lambda: moe.moe_balance_loss(l.double(), i, 1.0), lambda: moe.moe_balance_loss(l, i.long(), 1.0),
                lambda: moe.moe_balance_loss(l, i, 1.0, seq_len=3), lambda: moe.moe_balance_loss(l, i, 1.0, seq_len=0),
                lambda: moe.moe_balance_loss(l, i, 1.0, mask=torch.ones(7, dtype=torch.uint8, device="cuda")),
                lambda: moe.moe_balance_loss(l, i[:4].contiguous(), 1.0)):
        with pytest.raises(ValueError):
            bad()
    _, c, n = moe.moe_balance_loss(l, i, 1.0)
    with pytest.raises(ValueError):
        moe.moe_balance_loss_bwd(l, c, n, 2, 1.0, seq_len=4)   # another split than the counts'
    with pytest.raises(ValueError):
        moe.moe_balance_loss_bwd(l, c, n, 2, 1.0, d_logits_in=torch.zeros((8, 5), device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.moe_balance_loss_bwd(l, c, n, 5, 1.0)              # k > E
