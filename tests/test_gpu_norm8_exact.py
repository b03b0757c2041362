"""The norm to MXFP8 rows where its results are known to (almost) the last bit.

The product s r w is rounded once, and little more: r is kept in two float32 words (s times the first is exact
for bf16 rows, and has a second word for float32 rows), and the sums of squares in float64 beside float32 sums of
eight. With integers of up to 255 those sums of eight are exact
(8 * 255^2 < 2^24). r is one Newton step in float64 from a float32 value off by at most 8 u (u = 2^-24: a
rounding each of the mean, the root and the quotient, correctly rounded or nearly): off by 1.5 (8 u)^2 < 2^-17 u.
The second words and their products with w add less than 2^-39. What is left is the product's own rounding:
u (1 + 2^-13) of the value in all."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev_bf16, host
from moe_inputs import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
ONCE = U * (1 + 2.0 ** -13)


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_expert_gemm_amd as g
    g.lib()
    return g


def _put(a, bf16):
    a = np.ascontiguousarray(a, np.float32)
    if bf16:
        b = f32_to_bf16_bits(a)
        return bf16_bits_to_f32(b).astype(np.float64), dev_bf16(b)
    return a.astype(np.float64), torch.from_numpy(a).cuda()


@pytest.mark.parametrize("T,H", [(40, 32), (33, 480), (20, 1056), (30, 2048), (9, 4128), (7, 8224), (12, 16384)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_product_is_rounded_about_once(moe, T, H, dtype):
    print(f"norm mxfp8 rounded once T={T} H={H} {dtype}", flush=True)
    g, bf16, eps = np.random.default_rng(T + H), dtype == "bf16", 2.0 ** -20
    xf, x = _put(g.integers(-127, 128, (T, H)), bf16)
    rf, res = _put(g.integers(-128, 129, (T, H)), bf16)
    wf, w = _put(np.exp2(g.integers(-3, 4, H)) * (1 + g.standard_normal(H) / 8), bf16)
    r = moe.moe_add_norm_mxfp8(x, w, residual=res, eps=eps, with_y=True, save_for_bwd=True)
    s = xf + rf
    assert np.array_equal(host(r["sum"]), s)
    rstd = 1 / np.sqrt((s * s).mean(1) + eps)
    n = s * rstd[:, None] * wf
    err = np.abs(host(r["rstd"]) - rstd)
    assert np.all(err <= ONCE * rstd), f"rstd: {(err / rstd).max() / U:.3f} u"
    if not bf16:
        err = np.abs(host(r["y"]) - n)
        assert np.all(err <= ONCE * np.abs(n)), f"y: {(err / np.maximum(np.abs(n), 1e-30)).max() / U:.3f} u"
    else:
        assert np.all(np.abs(host(r["y"]) - n) <= (2.0 ** -8 + ONCE * (1 + 2.0 ** -8)) * np.abs(n))
    lo, hi, ok = oracle.mxfp8_bounds(n, ONCE * np.abs(n), host(r["scales"]))
    v = oracle.mxfp8_dequantize(host(r["codes"]), host(r["scales"]))
    assert ok.all() and np.all((lo <= v) & (v <= hi))


@pytest.mark.parametrize("H", [256, 2048, 8192])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_codes_of_exact_values(moe, H, dtype):
    """Rows of +-1 and +-3 with a mean square of 3 and eps = 1: r is 1/2 and n = s w / 2 exactly, so that codes and
    scales have one right answer: halfway values, subnormal codes, largest magnitudes at and just above 1.75 * 2^n."""
    g, bf16, T = np.random.default_rng(H), dtype == "bf16", 24
    s = np.ones((T, H))
    for t in range(T):  # the threes, a quarter of the row, stay out of every other block
        free = np.flatnonzero(np.arange(H) // 32 % 2 == 0)
        s[t, g.choice(free, H // 4, replace=False)] = 3.0
    s *= g.choice([-1.0, 1.0], (T, H))
    w = np.empty((H // 32, 32))
    for i in range(H // 32):
        e, kind = float(g.integers(-100, 100)), i // 2 % 4
        if kind == 0:
            w[i] = (2 * g.integers(8, 16, 32) + 1) / 16 * np.exp2(e + g.integers(-4, 1, 32))
        elif kind == 1:
            w[i] = (2 * g.integers(0, 9, 32) + 1) * np.exp2(e - 10)
            w[i, int(g.integers(0, 32))] = 256 * np.exp2(e)
        else:
            w[i] = g.uniform(0, 1.7, 32) * np.exp2(e)
            w[i, int(g.integers(0, 32))] = (1.75 if kind == 2 else 1.7578125) * np.exp2(e)
    sf, x = _put(s, bf16)
    wf, wt = _put(f32_to_bf16_f(w.reshape(H)), bf16)
    r = moe.moe_add_norm_mxfp8(x, wt, eps=1.0, with_y=True, save_for_bwd=True)
    assert bool((r["rstd"] == 0.5).all())
    n = sf * 0.5 * wf
    codes, scales = oracle.mxfp8_quantize(n)
    assert np.array_equal(host(r["scales"]), scales), "scales"
    assert np.array_equal(host(r["codes"]), codes), "codes"
    if not bf16:
        assert np.array_equal(host(r["y"]), n)


def f32_to_bf16_f(a):
    """values rounded to bf16: products with 1/2 and 3/2 are then exact in float32"""
    return bf16_bits_to_f32(f32_to_bf16_bits(np.ascontiguousarray(a, np.float32)))


@pytest.mark.parametrize("H", [512, 4096, 16384])
def test_codes_next_to_a_border(moe, H):
    """Products within a float32 step or two of the middle between two codes, on either side: the codes are
    those of the product, not of its float32 rounding, which often is the middle itself. Known to 2^-40: r to
    1.5 (8 u)^2 < 2^-41, the second words to a few u^2 each."""
    g, eps = np.random.default_rng(H), 2.0 ** -20
    wrong_after_rounding = 0
    for _ in range(4):
        s = g.integers(1, 256, (1, H)).astype(np.float64) * g.choice([-1.0, 1.0], (1, H))
        rstd = 1 / np.sqrt((s * s).mean() + eps)
        middle = (2 * g.integers(8, 16, H) + 1) / 16 * np.exp2(g.integers(-2, 1, H))
        wf, w = _put(middle / (np.abs(s[0]) * rstd) * (1 + U * g.integers(-1, 2, H)), False)
        n = s * rstd * wf
        _, x = _put(s, False)
        r = moe.moe_add_norm_mxfp8(x, w, eps=eps, with_y=True)
        lo, hi, ok = oracle.mxfp8_bounds(n, 2.0 ** -40 * np.abs(n), host(r["scales"]))
        v = oracle.mxfp8_dequantize(host(r["codes"]), host(r["scales"]))
        assert ok.all() and np.all((lo <= v) & (v <= hi)), f"{int(((v < lo) | (v > hi)).sum())} of {H} codes"
        assert np.all(np.abs(host(r["y"]) - n) <= ONCE * np.abs(n))          # y is rounded to nearest
        lo, hi, _ = oracle.mxfp8_bounds(n.astype(np.float32).astype(np.float64), 0 * n, host(r["scales"]))
        wrong_after_rounding += int((lo != v).sum())
    assert wrong_after_rounding > H // 16      # the inputs are what they are meant to be


def test_bf16_output_next_to_a_border(moe):
    """A bf16 y is the product rounded once: half a bf16 step off, and 2^-38 for what the product is known to (r's
    second word, and its product with w, are each rounded 2^-16 below: 2^-40 and 2^-40, and r's 2^-41)."""
    g, eps = np.random.default_rng(3), 2.0 ** -20
    for H in (2048, 8192, 16384):
        sf, x = _put(g.integers(-255, 256, (64, H)), True)
        wf, w = _put(1 + 0.2 * g.standard_normal(H), True)
        y = host(moe.moe_add_norm_mxfp8(x, w, eps=eps, with_y=True)["y"])
        n = sf / np.sqrt((sf * sf).mean(1, keepdims=True) + eps) * wf
        half = np.exp2(np.floor(np.log2(np.maximum(np.abs(n), 1e-30))) - 8)
        assert np.all(np.abs(y - n) <= half + 2.0 ** -38 * np.abs(n))
