"""GPU parity of the residual add + norm to MXFP8 rows and of the reading of MXFP8 rows, against
the float64 oracle.

Tolerances (u = 2^-24, float32's half step; h = the stored type's: 2^-8 for bf16): the sum adds at
most 17 float32 terms, each addition off by u of the magnitudes added so far: 17 u of the sum of
magnitudes, and h of the value for its one rounding. The norm is compared on the device's own
stored sum: the mean of squares adds positive terms, at most 64 a thread in a row, then over lanes
and wavefronts: r is off by at most 64 u relative, a product of it by 70 u, with y's rounding h. A
code may be any that a value within 70 u of the exact one rounds to: rounding is monotone, so
these are the codes between those of the interval's ends. Reading is exact."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev_bf16, host
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


def _put(a, bf16):
    """(float64 values as stored, device tensor)"""
    a = np.ascontiguousarray(a, np.float32)
    if bf16:
        b = f32_to_bf16_bits(a)
        return bf16_bits_to_f32(b).astype(np.float64), dev_bf16(b)
    return a.astype(np.float64), torch.from_numpy(a).cuda()


def _check(r, sum_ref, sum_mag, w, bf16, codes_only=False):
    half = 2.0 ** -8 if bf16 else U
    s = host(r["sum"]).astype(np.float64)
    assert np.all(np.abs(s - sum_ref) <= half * np.abs(sum_ref) + 17 * U * sum_mag + 1e-40), "sum"
    rstd = 1 / np.sqrt((s * s).mean(1) + EPS)
    n = s * rstd[:, None] * w
    if "rstd" in r:
        assert np.all(np.abs(host(r["rstd"]) - rstd) <= 70 * U * rstd), "rstd"
    if "y" in r:
        assert np.all(np.abs(host(r["y"]) - n) <= (half + 70 * U) * np.abs(n) + 1e-40), "y"
    scales = host(r["scales"])
    lo, hi, ok = oracle.mxfp8_bounds(n, 70 * U * np.abs(n), scales)
    assert ok.all(), "scale bytes"
    v = oracle.mxfp8_dequantize(host(r["codes"]), scales)
    assert np.all((lo <= v) & (v <= hi)), "codes"


# rows of one wavefront and of teams, widths that leave lanes of a team idle, the widest
@pytest.mark.parametrize("T,H", [(1, 32), (3, 64), (5, 480), (7, 512), (9, 544), (4, 1024), (6, 1056), (2, 2048), (3, 2080),
                                 (5, 4096), (2, 4128), (3, 8192), (2, 8224), (2, 16384), (1100, 2048), (2500, 96),
                                 (2100, 4160), (9000, 32)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_residual_and_norm(moe, T, H, dtype):
    print(f"add norm mxfp8 T={T} H={H} {dtype}", flush=True)
    g, bf16 = np.random.default_rng(T * 7 + H), dtype == "bf16"
    xf, x = _put(g.standard_normal((T, H)) * np.exp2(g.integers(-9, 9, (T, 1))), bf16)
    rf, res = _put(g.standard_normal((T, H)), bf16)
    wf, w = _put(1 + 0.2 * g.standard_normal(H), bf16)
    r = moe.moe_add_norm_mxfp8(x, w, residual=res, eps=EPS, with_y=True, save_for_bwd=True)
    _check(r, xf + rf, np.abs(xf) + np.abs(rf), wf, bf16)
    alone = moe.moe_add_norm_mxfp8(x, w, eps=EPS)
    assert alone["sum"] is x and set(alone) == {"sum", "codes", "scales"}
    _check(alone, xf, np.abs(xf), wf, bf16)


@pytest.mark.parametrize("T,H,k", [(1, 2048, 8), (5, 64, 2), (33, 512, 3), (7, 1056, 16), (2, 8192, 5), (1500, 256, 2),
                                   (1200, 2048, 8), (3, 16384, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_combined_rows(moe, T, H, k, dtype):
    print(f"add norm mxfp8 combine T={T} H={H} k={k} {dtype}", flush=True)
    g, bf16 = np.random.default_rng(T * 7 + H + k), dtype == "bf16"
    xf, x = _put(g.standard_normal((T * k, H)), bf16)
    rf, res = _put(g.standard_normal((T, H)), bf16)
    wf, w = _put(1 + 0.2 * g.standard_normal(H), bf16)
    rows = g.permutation(T * k).astype(np.int32)
    rows[g.permutation(T * k)[:T * k // 5]] = -1
    if T > 1:
        rows[:k] = -1                  # a token whose every slot was dropped
        rows[k] = T * k                # out of range: adds nothing
    rmap, per = torch.from_numpy(rows).cuda(), rows.reshape(T, k)
    r = moe.moe_add_norm_mxfp8(x, w, residual=res, row_id_map=rmap, k=k, eps=EPS, with_y=True, save_for_bwd=True)
    _check(r, oracle.add_rows(xf, rf, per), oracle.add_rows(np.abs(xf), np.abs(rf), per), wf, bf16)
    r = moe.moe_add_norm_mxfp8(x, w, row_id_map=rmap, k=k, eps=EPS, with_y=True, save_for_bwd=True)
    _check(r, oracle.add_rows(xf, None, per), oracle.add_rows(np.abs(xf), None, per), wf, bf16)
    if T > 1:                          # the norm of a zero row: zero codes under the smallest scale
        assert not host(r["codes"])[0].any() and not host(r["scales"])[0].any()


def test_sum_written_over_its_inputs(moe):
    g = torch.Generator(device="cuda").manual_seed(3)
    for dt in (torch.bfloat16, torch.float32):
        x, res = (torch.randn((50, 1056), generator=g, device="cuda").to(dt) for _ in range(2))
        w = torch.ones(1056, dtype=dt, device="cuda")
        want = moe.moe_add_norm_mxfp8(x, w, residual=res, with_y=True)
        for name in ("res", "x"):
            a, b = x.clone(), res.clone()
            out = b if name == "res" else a
            got = moe.moe_add_norm_mxfp8(a, w, residual=b, with_y=True, out=out)
            assert got["sum"] is out
            for key in want:
                assert torch.equal(got[key], want[key]), (dt, name, key)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_that_are_not_finite(moe, dtype):
    """A row with an infinity or a NaN: every block whose norm is not finite carries the NaN scale and
    codes 0; the other rows are what they are without it."""
    g, bf16 = np.random.default_rng(11), dtype == "bf16"
    H = 256
    xf, x = _put(g.standard_normal((6, H)), bf16)
    wf, w = _put(1 + 0.2 * g.standard_normal(H), bf16)
    clean = moe.moe_add_norm_mxfp8(x, w, eps=EPS)
    x[1, 5], x[3, 40], x[4, 100] = float("inf"), float("nan"), -float("inf")
    r = moe.moe_add_norm_mxfp8(x, w, eps=EPS, with_y=True)
    y, s, c = host(r["y"]), host(r["scales"]), host(r["codes"])
    bad = ~np.isfinite(y).reshape(6, H // 32, 32).all(2)
    assert bad[[1, 3, 4]].any(1).all() and not bad[[0, 2, 5]].any()
    assert (s[bad] == 255).all() and not c.reshape(6, -1, 32)[bad].any() and (s[~bad] < 255).all()
    for t in (0, 2, 5):
        assert torch.equal(r["codes"][t], clean["codes"][t]) and torch.equal(r["scales"][t], clean["scales"][t])
    assert np.array_equal(np.isnan(host(moe.mxfp8_dequantize(r["codes"], r["scales"]))).reshape(6, -1, 32), bad[:, :, None].repeat(32, 2))


def test_smallest_and_largest_magnitudes(moe):
    """Rows near both ends of float32: squares that vanish beside eps, weights that take n far up and down."""
    H = 64
    for scale, wscale in ((2.0 ** -60, 1.0), (2.0 ** -126, 1.0), (1.0, 2.0 ** -100), (1.0, 2.0 ** 100), (2.0 ** 60, 2.0 ** -40)):
        g = np.random.default_rng(5)
        xf, x = _put(scale * g.standard_normal((8, H)), False)
        wf, w = _put(wscale * (1 + 0.1 * g.standard_normal(H)), False)
        r = moe.moe_add_norm_mxfp8(x, w, eps=EPS)
        rstd = 1 / np.sqrt((xf * xf).mean(1) + EPS)
        n = xf * rstd[:, None] * wf
        # the product s r is rounded to a multiple of 2^-149 before w multiplies it, and the result again
        err = 70 * U * np.abs(n) + 2.0 ** -149 * (1 + np.abs(wf))
        lo, hi, ok = oracle.mxfp8_bounds(n, err, host(r["scales"]))
        v = oracle.mxfp8_dequantize(host(r["codes"]), host(r["scales"]))
        assert ok.all() and np.all((lo <= v) & (v <= hi)), (scale, wscale)


def test_read_every_code_and_scale(moe):
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1).cuda()          # row s: every code under scale byte s
    scales = torch.arange(256, dtype=torch.uint8).repeat_interleave(8).reshape(256, 8).cuda()
    got = host(moe.mxfp8_dequantize(codes, scales))
    ref = oracle.mxfp8_dequantize(codes.cpu().numpy(), scales.cpu().numpy())
    ref[255] = np.nan
    with np.errstate(over="ignore"):
        want = bf16_bits_to_f32(f32_to_bf16_bits(np.where(np.isnan(ref), 0, ref).astype(np.float32))).astype(np.float64)
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan)
    assert np.array_equal(got[~nan], want[~nan])
    assert np.array_equal(np.signbit(got[~nan]), np.signbit(ref[~nan]))


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (77, 1440), (5, 16384), (4000, 64), (1 << 16, 32)])
def test_read_rows(moe, rows, cols):
    print(f"read mxfp8 {rows} x {cols}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    codes = torch.randint(0, 127, (rows, cols), generator=g, device="cuda").to(torch.uint8)
    scales = torch.randint(90, 160, (rows, cols // 32), generator=g, device="cuda").to(torch.uint8)
    ref = torch.from_numpy(oracle.mxfp8_dequantize(codes.cpu().numpy(), scales.cpu().numpy())).to(torch.bfloat16)
    got = moe.mxfp8_dequantize(codes, scales)
    assert torch.equal(got.cpu(), ref)
    n = 2 * rows + 3
    src = torch.randint(0, rows, (n,), generator=g, device="cuda").int()
    src[0], src[n // 2], src[-1] = -1, rows, 2 ** 31 - 1                        # left as they were
    out = torch.full((n, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    assert moe.mxfp8_dequantize(codes, scales, src_row=src, out=out) is out
    want = torch.full((n, cols), 7.0, dtype=torch.bfloat16)
    at = src.cpu().long()
    ok = (at >= 0) & (at < rows)
    want[ok] = ref[at[ok]]
    assert torch.equal(out.cpu(), want)


def test_read_shapes_of_no_rows(moe):
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    assert moe.mxfp8_dequantize(z(0, 64), z(0, 2)).shape == (0, 64)
    assert moe.mxfp8_dequantize(z(2, 3, 64), z(2, 3, 2)).shape == (2, 3, 64)
    out = torch.full((3, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    src = torch.zeros(3, dtype=torch.int32, device="cuda")
    moe.mxfp8_dequantize(z(0, 64), z(0, 2), src_row=src, out=out)               # no row to read: none written
    assert bool((out == 2.0).all())
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    r = moe.moe_add_norm_mxfp8(x, torch.ones(64, dtype=torch.bfloat16, device="cuda"), residual=x, save_for_bwd=True)
    assert r["codes"].shape == (0, 64) and r["rstd"].shape == (0,)


def test_refusals(moe):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    m = torch.zeros(4, dtype=torch.int32, device="cuda")
    bad = [dict(weight=w.float()), dict(residual=x.float()), dict(residual=x[:3].contiguous()), dict(k=2), dict(k=0),
           dict(row_id_map=m, k=3), dict(row_id_map=m.long()), dict(weight=w[:32].contiguous()), dict(out=x.float()),
           dict(x=x.t()), dict(residual=x.cpu())]
    for kw in bad:
        with pytest.raises(ValueError):
            moe.moe_add_norm_mxfp8(**{"x": x, "weight": w, **kw})
    with pytest.raises(moe.MoeError, match="H % 32"):
        moe.moe_add_norm_mxfp8(x[:, :48].contiguous(), w[:48].contiguous())
    with pytest.raises(moe.MoeError, match="eps"):
        moe.moe_add_norm_mxfp8(x, w, eps=0.0)
    with pytest.raises(moe.MoeError, match="aligned"):
        moe.moe_add_norm_mxfp8(torch.zeros(4 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 64), w)
    c, s = (torch.zeros((4, n), dtype=torch.uint8, device="cuda") for n in (64, 2))
    for kw in (dict(scales=s[:3].contiguous()), dict(codes=c.int()), dict(src_row=m.long()), dict(src_row=m.view(2, 2)),
               dict(out=x.float()), dict(src_row=m[:2].contiguous(), out=x), dict(codes=c.view(2, 2, 64), scales=s.view(2, 2, 2), src_row=m)):
        with pytest.raises(ValueError):
            moe.mxfp8_dequantize(**{"codes": c, "scales": s, **kw})
