"""The MXFP4 oracle: the codebook, the scale rule and ties by exhaustive and closed-form
checks (CPU)."""
import numpy as np
import pytest

import oracle


def test_codes_read_back_as_themselves():
    """Every E2M1 value next to the largest one (so the scale is fixed) codes to itself."""
    for s in (-20, 0, 7):
        block = np.zeros((1, 32))
        block[0, :16] = np.concatenate([oracle.E2M1_VALUES, -oracle.E2M1_VALUES]) * 2.0 ** s
        codes, scales = oracle.mxfp4_encode(block)
        assert scales[0, 0] == s + 127 and codes[0, :16].tolist() == list(range(16))
        assert np.array_equal(oracle.mxfp4_dequantize(oracle.mxfp4_pack(codes), scales), block)


def test_midpoints_go_to_the_even_code():
    mids = (oracle.E2M1_VALUES[1:] + oracle.E2M1_VALUES[:-1]) / 2
    block = np.full((1, 32), 6.0)
    block[0, :7] = mids
    block[0, 7:14] = np.nextafter(mids, 0)
    block[0, 14:21] = np.nextafter(mids, 10)
    codes = oracle.mxfp4_encode(block)[0][0]
    assert codes[:7].tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert codes[7:14].tolist() == list(range(7)) and codes[14:21].tolist() == list(range(1, 8))


@pytest.mark.parametrize("seed", range(3))
def test_scale_is_the_smallest_that_fits(seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((40, 64)) * 2.0 ** rng.integers(-30, 30, (40, 1))
    _, scales = oracle.mxfp4_encode(x)
    s = scales.astype(int) - 127
    amax = np.abs(x.reshape(40, 2, 32)).max(-1)
    assert np.all(amax <= 6 * 2.0 ** s) and np.all(amax > 6 * 2.0 ** (s - 1.0))
    # nothing is further off than half the widest step around it
    err = np.abs(oracle.mxfp4_qdq(x) - x).reshape(40, 2, 32)
    assert np.all(err <= 2.0 ** s[..., None])


def test_zero_signs_limits_and_not_finite():
    x = np.zeros((5, 32))
    x[0, 3] = -0.0
    x[1, 0] = 2.0 ** -140        # below the smallest scale's step
    x[2, 0] = 2.0 ** 127 * 1.9   # bf16's range
    x[3, 5], x[4, 6] = np.inf, np.nan
    codes, scales = oracle.mxfp4_encode(x)
    assert scales[:, 0].tolist() == [0, 0, 127 + 125 + 1, 255, 255]
    assert codes[0, 3] == 8 and codes[1, 0] == 0 and codes[3].max() == 0
    assert np.all(np.isnan(oracle.mxfp4_qdq(x)[3:]))


def test_mlp_on_exact_operands_is_the_plain_one():
    """Operands that MXFP4 holds exactly, and h left unquantised: the plain SwiGLU MLP."""
    rng = np.random.default_rng(1)
    x = rng.choice(oracle.E2M1_VALUES, (6, 32))
    x[:, 0] = 6
    w1 = rng.choice(oracle.E2M1_VALUES, (2, 64, 32)) * 0.125
    w2 = rng.choice(oracle.E2M1_VALUES, (2, 32, 32)) * 0.125
    off, p = np.array([0, 2, 6]), rng.uniform(0.1, 1, 6)
    y, h = oracle.mxfp4_mlp_forward(x, w1, w2, off, p, h_quantise=lambda v: v)
    for e in range(2):
        r = slice(off[e], off[e + 1])
        g, u = x[r] @ w1[e, :32].T, x[r] @ w1[e, 32:].T
        assert np.allclose(h[r], g / (1 + np.exp(-g)) * u * p[r, None])
        assert np.allclose(y[r], h[r] @ w2[e].T)
