"""GPU parity of MXFP4: the quantiser bit for bit, the grouped products and the grouped MLP
against the float64 oracle.

Tolerances: products of two E2M1 codes and their scales are exact in float32, so a product
is off by its sums alone. An MFMA adds 64 or 128 products to its accumulator with at most a
few float32 roundings; K / 64 + 8 roundings of the sum of magnitudes cover the chain, the
wavefronts' partial sums and the zero steps. The bf16 result is off by another half step
(2^-8). In the MLP an h that lies within its own float32 error of a code's border may take
either code: the allowance is the difference between the quantised h + and - that error."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev_bf16, host
from moe_inputs import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_expert_gemm_amd as g
    g.lib()
    return g


def _bf16(a):
    b = f32_to_bf16_bits(np.ascontiguousarray(a, np.float32))
    return bf16_bits_to_f32(b).astype(np.float64), dev_bf16(b)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ---------------------------------------------------------------------------
# quantisation
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (17, 256), (129, 1056), (2048, 4096), (70001, 32)])
def test_quantize_bit_exact(moe, rows, cols):
    rng = np.random.default_rng(rows + cols)
    f, t = _bf16(rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-12, 12, (rows, 1)))
    codes, scales = moe.mxfp4_quantize(t)
    rc, rs = oracle.mxfp4_quantize(f)
    assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(scales.cpu().numpy(), rs)
    back = moe.mxfp4_dequantize(codes, scales)
    assert np.array_equal(host(back), oracle.mxfp4_dequantize(rc, rs))


def test_quantize_every_border(moe):
    """Every bf16 value from 2^-4 to 8 beside a 6 (scale 1), its negatives, ties included; blocks
    whose maximum lies at and around 6 * 2^s; zeros of both signs; the type's extremes; and
    infinities and NaN, whose blocks are NaN as a whole."""
    bits = np.arange(0x3D80, 0x4100, dtype=np.uint16)
    vals = bf16_bits_to_f32(bits).astype(np.float64)
    vals = vals[vals <= 6]
    vals = np.concatenate([vals, -vals, [0.0, -0.0]])
    n = -(-vals.size // 31)
    x = np.zeros((n, 32))
    x[:, 1:].flat[:vals.size] = vals
    x[:, 0] = 6
    edge = np.zeros((64, 32))
    m = bf16_bits_to_f32(np.array([0x40BF, 0x40C0, 0x40C1, 0x4000], np.uint16)).astype(np.float64)  # around 6, and 2
    for i in range(64):
        edge[i, i % 32] = m[i % 4] * 2.0 ** (-120 + 4 * (i // 4)) * (-1) ** i
        edge[i, (i + 7) % 32] = m[(i + 1) % 4] * 2.0 ** (-122 + 4 * (i // 4))
    lim = np.zeros((6, 32))
    lim[1] = -0.0
    lim[2, 3] = bf16_bits_to_f32(np.array([0x7F7F], np.uint16))[0]      # the largest bf16
    lim[3, 4] = bf16_bits_to_f32(np.array([0x0001], np.uint16))[0]      # the smallest
    lim[4, :] = bf16_bits_to_f32(np.array([0x0080], np.uint16))[0]      # the smallest normal one
    lim[5, 9] = -bf16_bits_to_f32(np.array([0x0041], np.uint16))[0]
    f, t = _bf16(np.concatenate([x, edge, lim]))
    codes, scales = moe.mxfp4_quantize(t)
    rc, rs = oracle.mxfp4_quantize(f)
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), rc)
    got, want = host(moe.mxfp4_dequantize(codes, scales)), oracle.mxfp4_dequantize(rc, rs)
    want = np.where(np.abs(want) > 3.4e38, np.copysign(np.inf, want), want)  # past bf16's range
    assert np.array_equal(got, want) and np.array_equal(np.signbit(got), np.signbit(want))
    bad = torch.ones((3, 64), dtype=torch.bfloat16, device="cuda")
    bad[0, 3], bad[1, 40], bad[2, 63] = float("nan"), float("inf"), -float("inf")
    codes, scales = moe.mxfp4_quantize(bad)
    assert scales.tolist() == [[255, 125], [125, 255], [125, 255]] and int(codes[0, :16].sum()) == 0
    back = moe.mxfp4_dequantize(codes, scales)
    assert torch.isnan(back[0, :32]).all() and torch.all(back[0, 32:] == 1) and torch.isnan(back[1:, 32:]).all()


def test_quantize_empty_and_refusals(moe):
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    c, s = moe.mxfp4_quantize(e)
    assert c.shape == (0, 32) and s.shape == (0, 2) and moe.mxfp4_dequantize(c, s).shape == (0, 64)
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    c, s = moe.mxfp4_quantize(x.view(2, 2, 64))
    assert c.shape == (2, 2, 32) and s.shape == (2, 2, 2)
    for bad in (lambda: moe.mxfp4_quantize(x.float()), lambda: moe.mxfp4_quantize(x.t()), lambda: moe.mxfp4_quantize(x.cpu()),
                lambda: moe.mxfp4_dequantize(c, s[:1]), lambda: moe.mxfp4_dequantize(c.int(), s)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(moe.MoeError):
        moe.mxfp4_quantize(x[:, :48].contiguous())


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

def _weights(rng, E, N, K, scale=0.02):
    """E weights as MXFP4: their values, codes and scales, block scales that differ widely."""
    w = scale * rng.standard_normal((E, N, K)) * 2.0 ** rng.integers(-3, 4, (E, N, K // 32)).repeat(32, axis=2)
    c, s = oracle.mxfp4_quantize(w)
    return oracle.mxfp4_dequantize(c, s), c, s


def _offsets(sizes):
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)


def _product_ref(xq, w, off):
    y, mag = np.zeros((xq.shape[0], w.shape[1])), np.zeros((xq.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        r = slice(off[e], off[e + 1])
        y[r], mag[r] = xq[r] @ w[e].T, np.abs(xq[r]) @ np.abs(w[e]).T
    return y, mag


def _steps(K):
    return (K / 64 + 8) * U


LINEAR = [
    (256, 256, [1]),
    (256, 512, [0, 3, 0, 16, 17]),
    (768, 256, [5, 1, 0, 0, 2, 64, 65, 15]),
    (1280, 256, [128, 0, 129, 31]),
    (512, 768, [300, 1, 256, 257, 0]),
    (2816, 256, [40, 200]),
    (256, 256, [1] * 128),
    (1024, 512, [0] * 63 + [7] + [0] * 36 + [1]),
    (512, 256, [0, 1500, 0, 513]),
    # 16 rows in all and one more: quantised by the product's own kernel, and before it
    (768, 512, [0, 5, 1, 0, 7]),
    (2816, 256, [6, 0, 8]),
    # every number of K steps modulo the tile kernel's ring, one step alone among them
    (256, 256, [300]),
    (768, 512, [70, 400]),
    (1024, 256, [513, 64]),
    (1536, 256, [0, 255, 256, 1]),
    (2304, 256, [200]),
]


@pytest.mark.parametrize("K,N,sizes", LINEAR)
@pytest.mark.parametrize("codes", [False, True])
def test_linear(moe, K, N, sizes, codes):
    rng = np.random.default_rng(K + N + sum(sizes))
    E, R = len(sizes), sum(sizes)
    print(f"mxfp4 linear K={K} N={N} E={E} R={R} codes={codes}", flush=True)
    off = _offsets(sizes)
    w, wc, ws = _weights(rng, E, N, K)
    spare = 3  # rows behind the last expert's: left as they were
    xf, x = _bf16(rng.standard_normal((R + spare, K)) * 2.0 ** rng.integers(-3, 4, (R + spare, K // 32)).repeat(32, axis=1))
    y = torch.full((R + spare, N), 5.0, dtype=torch.bfloat16, device="cuda")
    if codes:
        xc, xs = moe.mxfp4_quantize(x)
        got = moe.moe_grouped_linear_mxfp4(xc, _dev(wc), _dev(ws), _dev(off), x_scale=xs, out=y)
    else:
        got = moe.moe_grouped_linear_mxfp4(x, [_dev(a) for a in wc], [_dev(a) for a in ws], _dev(off), out=y)
    ref, mag = _product_ref(oracle.mxfp4_qdq(xf), w, off)
    g = host(got)
    assert np.all(g[R:] == 5.0)
    tol = 2.0 ** -8 * np.abs(ref[:R]) + _steps(K) * mag[:R] + 1e-38
    bad = np.abs(g[:R] - ref[:R]) / tol
    assert np.all(bad <= 1), (float(bad.max()), np.unravel_index(bad.argmax(), bad.shape))
    again = moe.moe_grouped_linear_mxfp4(x, _dev(wc), _dev(ws), _dev(off))
    assert torch.equal(again[:R], got[:R])


@pytest.mark.parametrize("sizes", [[3, 2], [40, 30], [300, 200]])
def test_linear_rows_before_the_first_expert(moe, sizes):
    """Expert e owns the rows [offsets[e], offsets[e + 1]): those before offsets[0] are left as they were."""
    rng = np.random.default_rng(sum(sizes))
    K, N, R, lead = 256, 256, sum(sizes) + 10, 10
    print(f"mxfp4 linear, {lead} rows before the first expert's {sizes}", flush=True)
    off = _offsets(sizes) + lead
    w, wc, ws = _weights(rng, 2, N, K)
    xf, x = _bf16(rng.standard_normal((R, K)))
    y = torch.full((R, N), 5.0, dtype=torch.bfloat16, device="cuda")
    g = host(moe.moe_grouped_linear_mxfp4(x, _dev(wc), _dev(ws), _dev(off.astype(np.int32)), out=y))
    ref, mag = _product_ref(oracle.mxfp4_qdq(xf), w, off)
    assert np.all(g[:lead] == 5.0)
    assert np.all(np.abs(g[lead:] - ref[lead:]) <= 2.0 ** -8 * np.abs(ref[lead:]) + _steps(K) * mag[lead:] + 1e-38)


def test_linear_not_finite_stays_in_its_rows_and_columns(moe):
    """An x row with a NaN gives a NaN row; a weight row whose scale byte is 255 a NaN column for
    that expert's rows; everything else is what it was."""
    rng = np.random.default_rng(4)
    K, N, sizes = 512, 256, [20, 300]
    off = _dev(_offsets(sizes))
    _, wc, ws = _weights(rng, 2, N, K)
    _, x = _bf16(rng.standard_normal((320, K)))
    base = moe.moe_grouped_linear_mxfp4(x, _dev(wc), _dev(ws), off)
    x2, ws2 = x.clone(), ws.copy()
    x2[7, 100] = float("nan")
    x2[200, 511] = float("inf")
    ws2[1, 33, 5] = 255
    y = moe.moe_grouped_linear_mxfp4(x2, _dev(wc), _dev(ws2), off)
    nan = torch.zeros((320, N), dtype=torch.bool, device="cuda")
    nan[7], nan[200], nan[20:, 33] = True, True, True
    assert torch.equal(torch.isnan(y), nan) and torch.equal(y[~nan], base[~nan])


# ---------------------------------------------------------------------------
# the grouped MLP
# ---------------------------------------------------------------------------

def _mlp_tolerance(xf, w1, w2, off, prob):
    """The oracle's y and the bound on the GPU's error described at the top of this file."""
    y, h = oracle.mxfp4_mlp_forward(xf, w1, w2, off, prob)
    xq = oracle.mxfp4_qdq(xf)
    H, I = xq.shape[1], h.shape[1]
    tol = np.zeros(y.shape)
    for e in range(w1.shape[0]):
        r = slice(off[e], off[e + 1])
        if off[e + 1] == off[e]:
            continue
        z, zm = xq[r] @ w1[e].T, np.abs(xq[r]) @ np.abs(w1[e]).T * _steps(H)
        g, u, dg, du = z[:, :I], z[:, I:], zm[:, :I], zm[:, I:]
        sg = 1 / (1 + np.exp(-g))
        silu = g * sg
        # |silu'| <= 1.1; the activation's own arithmetic: 16 roundings (exp's argument included: |g| u)
        dh = np.abs(prob[r, None]) * (1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du) + (16 + np.abs(g)) * U * np.abs(h[r])
        hi = np.copysign(np.abs(h[r]) + dh, h[r])
        lo = np.copysign(np.maximum(np.abs(h[r]) - dh, 0), h[r])
        slack = np.abs(oracle.mxfp4_qdq(hi) - oracle.mxfp4_qdq(lo))
        hq = np.abs(oracle.mxfp4_qdq(h[r]))
        tol[r] = slack @ np.abs(w2[e]).T + _steps(I) * (hq @ np.abs(w2[e]).T)
    return y, 2.0 ** -8 * np.abs(y) + tol + 1e-38


MLP = [
    (256, 256, [1]),
    (512, 256, [0, 2, 1, 0, 33]),
    (256, 768, [16, 17, 64, 65, 0, 1]),
    (768, 512, [130, 0, 257, 70]),
    (256, 256, [1] * 100 + [0] * 28),
    (512, 512, [900, 3]),
    (1024, 1280, [300, 129]),
    (1280, 768, [3, 0, 12, 1]),
    (512, 768, [17]),
    (1280, 256, [520]),
]


@pytest.mark.parametrize("H,I,sizes", MLP)
@pytest.mark.parametrize("act,wt", [("bf16", "codes"), ("codes", "codes"), ("bf16", "bf16")])
def test_mlp(moe, H, I, sizes, act, wt):
    rng = np.random.default_rng(H + I + sum(sizes))
    E, R = len(sizes), sum(sizes)
    print(f"mxfp4 mlp H={H} I={I} E={E} R={R} act={act} wt={wt}", flush=True)
    off = _offsets(sizes)
    if wt == "bf16":
        f1, t1 = _bf16(0.05 * rng.standard_normal((E, 2 * I, H)))
        f2, t2 = _bf16(0.05 * rng.standard_normal((E, H, I)))
        w1, w2, s1, s2 = oracle.mxfp4_qdq(f1), oracle.mxfp4_qdq(f2), None, None
    else:
        w1, c1, s1 = _weights(rng, E, 2 * I, H, 0.05)
        w2, c2, s2 = _weights(rng, E, H, I, 0.05)
        t1, t2, s1, s2 = _dev(c1), _dev(c2), _dev(s1), _dev(s2)
    xf, x = _bf16(rng.standard_normal((R, H)))
    prob = rng.uniform(0.05, 1.0, R).astype(np.float32)
    prob[0] = 0.0
    xs = None
    if act == "codes":
        x, xs = moe.mxfp4_quantize(x)
    y = moe.moe_grouped_mlp_fwd(x, t1, t2, _dev(off), _dev(prob), compute="mxfp4", x_perm_scale=xs, w_gate_up_scale=s1,
                                w_down_scale=s2)
    ref, tol = _mlp_tolerance(xf, w1, w2, off, prob.astype(np.float64))
    bad = np.abs(host(y) - ref) / tol
    assert np.all(bad <= 1), (float(bad.max()), np.unravel_index(bad.argmax(), bad.shape))
    assert torch.all(y[0] == 0)


def test_permuted_codes_and_workspace(moe):
    """moe_permute gathers MXFP4 rows with their scales (fresh and with the maps given), so that
    quantising T tokens and gathering codes equals gathering bf16 and quantising T*k rows; a
    caller's workspace, larger than needed and full of NaN bytes, serves too."""
    rng = np.random.default_rng(8)
    T, H, I, E, k = 70, 512, 256, 6, 3
    _, x = _bf16(rng.standard_normal((T, H)))
    _, c1, s1 = _weights(rng, E, 2 * I, H)
    _, c2, s2 = _weights(rng, E, H, I)
    w = [_dev(a) for a in (c1, c2, s1, s2)]
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    idx, prob = moe.moe_route_topk(logits, k)
    r = moe.moe_permute(x, idx, prob, E)
    xc, xs = moe.mxfp4_quantize(x)
    q = moe.moe_permute(xc, idx, prob, E, x_scale=xs)
    want = moe.mxfp4_quantize(r["x_perm"])
    assert torch.equal(q["x_perm"], want[0]) and torch.equal(q["x_perm_scale"], want[1])
    again = moe.moe_permute(xc, idx, None, E, x_scale=xs, row_id_map=r["row_id_map"])
    assert torch.equal(again["x_perm"], want[0]) and torch.equal(again["x_perm_scale"], want[1])
    a = moe.moe_grouped_mlp_fwd(r["x_perm"], w[0], w[1], r["offsets"], r["prob_perm"], compute="mxfp4",
                                w_gate_up_scale=w[2], w_down_scale=w[3])
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
    b = moe.moe_grouped_mlp_fwd(q["x_perm"], w[0], w[1], q["offsets"], q["prob_perm"], compute="mxfp4",
                                x_perm_scale=q["x_perm_scale"], w_gate_up_scale=w[2], w_down_scale=w[3], workspace=ws)
    assert torch.equal(a, b)


def test_no_rows_and_refusals(moe):
    E, H, I = 2, 256, 256
    w1 = torch.zeros((E, 2 * I, H // 2), dtype=torch.uint8, device="cuda")
    w2 = torch.zeros((E, H, I // 2), dtype=torch.uint8, device="cuda")
    s1 = torch.zeros((E, 2 * I, H // 32), dtype=torch.uint8, device="cuda")
    s2 = torch.zeros((E, H, I // 32), dtype=torch.uint8, device="cuda")
    off = torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda")
    x = torch.zeros((4, H), dtype=torch.bfloat16, device="cuda")
    p = torch.ones(4, device="cuda")
    none = torch.zeros(3, dtype=torch.int32, device="cuda")

    def mlp(x=x, w1=w1, w2=w2, s1=s1, s2=s2, off=off, p=p, **kw):
        return moe.moe_grouped_mlp_fwd(x, w1, w2, off, p, compute="mxfp4", w_gate_up_scale=s1, w_down_scale=s2, **kw)

    assert mlp(x=x[:0], off=none, p=p[:0]).shape == (0, H)
    out = torch.full((4, H), 3.0, dtype=torch.bfloat16, device="cuda")
    assert torch.all(mlp(off=none, out=out) == 3.0)       # no expert has rows: nothing is written
    assert moe.moe_grouped_linear_mxfp4(x[:0], w2, s2, none).shape == (0, H)
    for bad in (lambda: mlp(x=x.float()), lambda: mlp(x=x.cpu()), lambda: mlp(s1=None), lambda: mlp(s1=s1[:, :64].contiguous()),
                lambda: mlp(w1=w1[:1]), lambda: mlp(w2=w1), lambda: mlp(off=off.long()), lambda: mlp(off=off[:2]),
                lambda: mlp(p=p[:3]), lambda: mlp(x=torch.zeros((4, H // 2), dtype=torch.uint8, device="cuda")),
                lambda: mlp(out=out[:3]), lambda: mlp(w1=w1.transpose(1, 2)),
                lambda: moe.moe_grouped_linear_mxfp4(x, w2, None, off),
                lambda: moe.moe_grouped_linear_mxfp4(x, w2, s2, off, out=out.float())):
        with pytest.raises(ValueError):
            bad()
    odd = torch.zeros((2, 256, 160), dtype=torch.uint8, device="cuda")   # K = 320
    for bad in (lambda: mlp(save_for_bwd=True),
                lambda: moe.moe_grouped_linear_mxfp4(torch.zeros((4, 320), dtype=torch.bfloat16, device="cuda"), odd,
                                                     torch.zeros((2, 256, 10), dtype=torch.uint8, device="cuda"), off),
                lambda: moe.moe_grouped_mlp_bwd(x, x, torch.zeros((4, 2 * I), dtype=torch.bfloat16, device="cuda"), x, p,
                                                torch.zeros((E, 2 * I, H), dtype=torch.bfloat16, device="cuda"),
                                                torch.zeros((E, H, I), dtype=torch.bfloat16, device="cuda"), off,
                                                compute="mxfp4")):
        with pytest.raises(moe.MoeError):
            bad()
