"""GPU parity of the norms before and after the block, forward and backward, against the
float64 oracle.

Tolerances (u = 2^-24, float32's half step; h = the output type's: 2^-8 for bf16): an output
is rounded once (h of its value) on top of float32 arithmetic. The mean of squares is a sum
of positive terms added pairwise or in runs of at most 64, so r is off by at most 64 u
relative; a product of a few such factors by 80 u of the sum of the magnitudes it adds (the
combine's k <= 16 terms included). mean(dn n) is off by 64 u of the mean of |dn n|. A column
sum over T tokens adds runs of at most T / 512 + 4 tokens, then in each of 64 threads at most
the 2 T / 256 partial sums of its share, then 64 such sums, 4 at a time and then 16: 128 u of
the sum of magnitudes covers T <= 4096 (8 + 4 + 32 + 18, and a product's 4 roundings)."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import bf16_bits, dev_bf16, host
from moe_inputs import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_expert_gemm_amd as g
    g.lib()
    return g


class Maker:
    """Random tensors of one dtype: the float64 values and the device tensor."""

    def __init__(self, seed, dtype):
        self.rng, self.bf16 = np.random.default_rng(seed), dtype == "bf16"
        self.half = 2.0 ** -8 if self.bf16 else U

    def put(self, a):
        a = np.ascontiguousarray(a, np.float32)
        if self.bf16:
            b = f32_to_bf16_bits(a)
            return bf16_bits_to_f32(b).astype(np.float64), dev_bf16(b)
        return a.astype(np.float64), torch.from_numpy(a).cuda()

    def __call__(self, *shape, scale=1.0, mean=0.0):
        return self.put(mean + scale * self.rng.standard_normal(shape))


def _close(got, ref, mag, half, what):
    got = host(got).astype(np.float64)
    tol = half * np.abs(ref) + mag + 1e-40
    bad = np.abs(got - ref) / tol
    assert np.all(bad <= 1), f"{what}: {float(bad.max()):.2f} times the tolerance at {np.unravel_index(bad.argmax(), bad.shape)}"


def _gate(m, kind, T, H, group):
    if kind == "token":
        return m(T, mean=0.5, scale=0.3)
    if kind == "channel":
        return m(-(-T // group), H, mean=0.5, scale=0.3)
    return None, None


def _post(moe, m, T, H, k, kind, group, scale, next_norm, drop=0):
    xf, x = m(T, H)
    yf, y = m(T * k, H, scale=0.5)
    wf, w = m(H, mean=1.0, scale=0.2)
    w2f, w2 = m(H, mean=1.0, scale=0.2)
    gf, g = _gate(m, kind, T, H, group)
    rows = rmap = None
    if k > 1 or drop:
        rows = m.rng.permutation(T * k).astype(np.int32)
        rows[m.rng.permutation(T * k)[:drop]] = -1
        if drop >= k:
            rows[:k] = -1  # a token whose every slot was dropped
        rmap = torch.from_numpy(rows).cuda()
        rows = rows.reshape(T, k)
    r = moe.moe_post_norm(y, x, w, row_id_map=rmap, k=k, gate=g, gate_group=group if kind == "channel" else None,
                          residual_scale=scale, eps=EPS, save_for_bwd=True, next_weight=w2 if next_norm else None)
    ref, c, rr = oracle.post_norm(yf, xf, wf, EPS, rows, gf, group, scale)
    absc = np.abs(yf) if rows is None else oracle.post_norm(np.abs(yf), xf, wf, EPS, rows)[1]
    gg = np.abs(oracle.gate_rows(gf, group, T, H))
    mag = 80 * U * (np.abs(scale * xf) + gg * rr[:, None] * np.abs(wf) * absc)
    _close(r["out"], ref, mag, m.half, "out")
    _close(r["c"], c, 16 * U * absc, m.half, "c")
    rerr = (64 * U + 16 * U * (absc ** 2).sum(1) / ((c ** 2).sum(1) + H * EPS)) * rr
    assert np.all(np.abs(host(r["rstd"]) - rr) <= rerr)
    if next_norm:  # of the stored sum, bit for bit the separate call
        o = host(r["out"]).astype(np.float64)
        u, r2 = oracle.pre_norm(o, w2f, EPS)
        _close(r["y_next"], u, 80 * U * np.abs(u), m.half, "y_next")
        y2, rs2 = moe.moe_pre_norm(r["out"], w2, EPS, save_rstd=True)
        assert torch.equal(y2, r["y_next"]) and torch.equal(rs2, r["rstd_next"])
    # backward, on the stored sum and an exact r of it
    cf, cd = m.put(c)
    df, d = m(T, H)
    r32 = rr.astype(np.float32)
    sentinel = torch.full((T * k, H), 7.0, dtype=x.dtype, device="cuda")
    b = moe.moe_post_norm_bwd(d, cd, torch.from_numpy(r32).cuda(), w, row_id_map=rmap, k=k, gate=g,
                              gate_group=group if kind == "channel" else None, dy=sentinel)
    dc, dw, dg = oracle.post_norm_backward(df, cf, wf, r32, gf, group)
    a = np.abs(df * cf * r32[:, None])
    g_all = oracle.gate_rows(gf, group, T, H)
    dn = np.abs(df * g_all * wf)
    mag = 80 * U * r32[:, None] * (dn + np.abs(cf) * r32[:, None] * (dn * np.abs(cf) * r32[:, None]).mean(1, keepdims=True))
    got = host(b["dy"])
    if rows is None:
        _close(b["dy"], dc, mag, m.half, "dy")
    else:
        seen = np.zeros(T * k, bool)
        for j in range(k):
            ok = rows[:, j] >= 0
            seen[rows[ok, j]] = True
            tol = m.half * np.abs(dc[ok]) + mag[ok] + 1e-40
            assert np.all(np.abs(got[rows[ok, j]] - dc[ok]) <= tol), "dy"
        assert np.all(got[~seen] == 7.0), "a row without a slot was written"
    _close(b["dweight"], dw, 128 * U * (a * np.abs(g_all)).sum(0), U, "dweight")
    if kind == "token":
        _close(b["dgate"], dg, 80 * U * (a * np.abs(wf)).sum(1), U, "dgate")
    elif kind == "channel":
        mg = np.zeros(dg.shape)
        np.add.at(mg, np.arange(T) // group, a * np.abs(wf))
        _close(b["dgate"], dg, 128 * U * mg, U, "dgate")


# widths at the borders of the team sizes and of the 16-byte path, odd ones, one token
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,k,kind,group,scale,next_norm", [
    (1, 1, 1, "none", 1, 1.0, True),
    (1, 2048, 8, "none", 1, 1.0, True),
    (5, 8, 2, "token", 1, 0.5, False),
    (33, 510, 1, "channel", 7, 1.0, True),
    (70, 512, 2, "channel", 70, 2.0, False),
    (9, 513, 3, "token", 1, 1.0, True),
    (130, 520, 4, "channel", 1, 1.0, False),
    (64, 1024, 8, "channel", 3, 1.0, True),
    (21, 1027, 2, "channel", 21, -1.0, False),
    (700, 2048, 2, "channel", 350, 1.0, False),
    (2100, 96, 2, "channel", 700, 0.0, True),
    (1500, 131, 1, "channel", 9, 1.0, False),
    (3003, 24, 2, "channel", 13, 0.5, False),
    (40, 2056, 16, "token", 1, 1.0, True),
    (600, 4096, 2, "none", 1, 0.8, True),
    (18, 4104, 1, "channel", 18, 1.0, False),
    (6, 5001, 2, "channel", 2, 1.0, True),
    (12, 8192, 5, "token", 1, 1.0, False),
    (7, 16384, 2, "channel", 4, 1.0, True),
    (3, 16383, 1, "none", 1, 1.0, True),
])
def test_post_norm(moe, dtype, T, H, k, kind, group, scale, next_norm):
    print(f"post norm {dtype} T={T} H={H} k={k} gate={kind}/{group}", flush=True)
    _post(moe, Maker(T * 31 + H, dtype), T, H, k, kind, group, scale, next_norm)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_post_norm_dropped_slots(moe, dtype):
    """Slots that were dropped (-1) add nothing and get no gradient; a token left with none
    normalises to zero and stays finite."""
    print(f"post norm dropped {dtype}", flush=True)
    _post(moe, Maker(5, dtype), 50, 264, 4, "token", 1, 1.0, True, drop=60)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 100), (257, 512), (64, 999), (1500, 1024), (900, 2048), (2, 3000), (17, 4096),
                                 (5, 8200), (4, 16384)])
def test_pre_norm(moe, dtype, T, H):
    print(f"pre norm {dtype} T={T} H={H}", flush=True)
    m = Maker(T * 17 + H, dtype)
    xf, x = m(T, H)
    wf, w = m(H, mean=1.0, scale=0.2)
    y, rstd = moe.moe_pre_norm(x, w, EPS, save_rstd=True)
    ref, r = oracle.pre_norm(xf, wf, EPS)
    _close(y, ref, 80 * U * np.abs(ref), m.half, "y")
    assert np.all(np.abs(host(rstd) - r) <= 64 * U * r)
    assert torch.equal(moe.moe_pre_norm(x, w, EPS), y)
    df, d = m(T, H)
    af, a = m(T, H)
    r32 = host(rstd).astype(np.float64)
    for dx_in, s in ((None, 1.0), (a, 0.75)):
        dx, dw = moe.moe_pre_norm_bwd(d, x, w, rstd, dx_in=dx_in, dx_in_scale=s)
        refx, refw = oracle.pre_norm_backward(df, xf, wf, r32, None if dx_in is None else af, s)
        n = np.abs(xf) * r32[:, None]
        dn = np.abs(df * wf)
        mag = 80 * U * (r32[:, None] * (dn + n * (dn * n).mean(1, keepdims=True)) + (0 if dx_in is None else np.abs(s * af)))
        _close(dx, refx, mag, m.half, "dx")
        _close(dw, refw, 128 * U * (np.abs(df) * n).sum(0), U, "dweight")
    got, _ = moe.moe_pre_norm_bwd(d, x, w, rstd, dx_in=a, dx_in_scale=0.75, dx=a)   # in place
    assert got.data_ptr() == a.data_ptr() and torch.equal(got, dx)


def test_rows_off_the_16_byte_grid_and_strange_values(moe):
    """Tensors that start 2 bytes off a 16-byte border take the one-element path and agree with
    the aligned ones; a row of zeros stays zero; huge and tiny rows, an infinity and a NaN stay
    within their own row."""
    m = Maker(3, "bf16")
    T, H = 40, 1024
    xf, x = m(T, H)
    wf, w = m(H, mean=1.0)
    x[3] = 0
    x[4] *= 2.0 ** 60
    x[5] *= 2.0 ** -60
    store = torch.empty(T * H + 1, dtype=torch.bfloat16, device="cuda")
    off = store[1:].view(T, H)
    off.copy_(x)
    y, y_off = moe.moe_pre_norm(x, w), moe.moe_pre_norm(off, w)
    ref = oracle.pre_norm(host(x), wf, 1e-6)[0]
    _close(y, ref, 80 * U * np.abs(ref), 2.0 ** -8, "aligned")
    _close(y_off, ref, 80 * U * np.abs(ref), 2.0 ** -8, "off the grid")
    assert torch.all(y[3] == 0)
    bad = x.clone()
    bad[10, 5] = float("nan")
    bad[11, 6] = float("inf")
    z = moe.moe_pre_norm(bad, w)
    keep = [t for t in range(T) if t not in (10, 11)]
    assert torch.equal(z[keep], y[keep]) and torch.isnan(z[10]).all() and torch.isnan(z[11, 6])


def test_in_place_residual_repeat_and_no_tokens(moe):
    m = Maker(9, "bf16")
    T, H, k = 300, 768, 2
    _, x = m(T, H)
    _, y = m(T * k, H)
    _, w = m(H, mean=1.0)
    _, g = m(3, H)
    rows = torch.randperm(T * k, device="cuda").int()
    a = moe.moe_post_norm(y, x, w, row_id_map=rows, k=k, gate=g, save_for_bwd=True)
    _, d = m(T, H)
    b1 = moe.moe_post_norm_bwd(d, a["c"], a["rstd"], w, row_id_map=rows, k=k, gate=g)
    b2 = moe.moe_post_norm_bwd(d, a["c"], a["rstd"], w, row_id_map=rows, k=k, gate=g)
    assert all(torch.equal(b1[n], b2[n]) for n in b1)
    x2 = x.clone()
    moe.moe_post_norm(y, x2, w, row_id_map=rows, k=k, gate=g, out=x2)
    assert torch.equal(x2, a["out"])
    e = torch.empty((0, H), dtype=torch.bfloat16, device="cuda")
    r = moe.moe_post_norm(e, e, w, save_for_bwd=True, next_weight=w)
    assert r["out"].shape == (0, H)
    b = moe.moe_post_norm_bwd(e, e, r["rstd"], w)
    dx, dw = moe.moe_pre_norm_bwd(e, e, w, r["rstd"])
    assert torch.all(b["dweight"] == 0) and torch.all(dw == 0) and dx.shape == (0, H)


def test_refusals(moe):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    r = torch.ones(4, device="cuda")
    m = torch.zeros(8, dtype=torch.int32, device="cuda")
    y = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: moe.moe_pre_norm(x.half(), w.half()), lambda: moe.moe_pre_norm(x, w.float()),
                lambda: moe.moe_pre_norm(x.t(), w), lambda: moe.moe_pre_norm(x.cpu(), w.cpu()),
                lambda: moe.moe_pre_norm(x, w[:32]), lambda: moe.moe_post_norm(y, x, w, k=2),
                lambda: moe.moe_post_norm(y, x, w, row_id_map=m[:4], k=2),
                lambda: moe.moe_post_norm(x, x, w, gate=w), lambda: moe.moe_post_norm(x, x, w, gate=y, gate_group=4),
                lambda: moe.moe_post_norm(x, x, w, gate=x, gate_group=0),
                lambda: moe.moe_post_norm(y, x, w, row_id_map=m.long(), k=2),
                lambda: moe.moe_post_norm_bwd(x, y, r, w), lambda: moe.moe_post_norm_bwd(x, x, r.double(), w),
                lambda: moe.moe_pre_norm_bwd(x, x, w, r, dx_in=y)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: moe.moe_pre_norm(x, w, eps=0.0), lambda: moe.moe_pre_norm(x, w, eps=float("nan")),
                lambda: moe.moe_post_norm(x, x, w, eps=-1.0),
                lambda: moe.moe_pre_norm(torch.zeros((1, 16385), device="cuda"), torch.ones(16385, device="cuda"))):
        with pytest.raises(moe.MoeError):
            bad()
