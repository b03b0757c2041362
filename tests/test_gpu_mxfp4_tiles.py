"""MXFP4 products whose workgroups take several tiles each, and the row kernel's weight pipeline
past its first units.

A tile's first loads are issued in the tile before it, so a call of many tiles has paths that a
call of one tile a workgroup has not. Every call here has more than 2 x 256 tiles of uneven
experts (some empty, some of a few rows, more than 64 of them in places) and is compared bit for bit
with calls of one expert each, of at most 256 tiles, so of one tile a workgroup on a card of 256
CUs: the sums of a row do not depend on the other rows. A sample of rows is held against the
float64 oracle with the tolerances of test_gpu_mxfp4.py."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import host
from test_gpu_mxfp4 import _mlp_tolerance, _offsets, _product_ref, _steps
from test_gpu_mxfp4 import test_linear as _linear
from test_gpu_mxfp4 import test_mlp as _mlp

pytestmark = pytest.mark.gpu
TAIL = 96  # rows behind the last expert's, so that a slice of 65 rows can start at any of them


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_expert_gemm_amd as g
    g.lib()
    return g


def _sizes(rng, E, rows):
    """E uneven experts of about `rows` rows in all: some empty, some of fewer rows than a tile"""
    n = (rows / E * 2.0 ** rng.uniform(-3, 1.5, E)).astype(int)
    n[rng.permutation(E)[:max(1, E // 8)]] = 0
    n[rng.permutation(E)[:max(1, E // 8)]] = rng.integers(1, 9)
    n[-1] = 257
    n[E // 2] = 0
    return n.tolist()


def _randn(g, *shape, scale=1.0):
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(torch.bfloat16)


def _weights(moe, g, E, N, K, scale):
    c = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.empty((E, N, K // 32), dtype=torch.uint8, device="cuda")
    for e in range(E):
        c[e], s[e] = moe.mxfp4_quantize(_randn(g, N, K, scale=scale))
    return c, s


def _one_expert(off, e):
    """slice of the rows of a call of expert e alone, its offsets: more than 64 rows, so that tiles are taken"""
    b, n = int(off[e]), int(off[e + 1] - off[e])
    return slice(b, b + max(n, 65)), torch.tensor([0, n], dtype=torch.int32, device="cuda"), n


def _sample(off, rng):
    """rows to hold against the oracle: first and last of some experts, and around a tile's border"""
    some = [e for e in range(len(off) - 1) if off[e + 1] > off[e]]
    picked = [some[0], some[-1], *rng.permutation(some)[:4].tolist()]
    rows = {}
    for e in sorted(set(picked)):
        b, n = int(off[e]), int(off[e + 1] - off[e])
        rows[e] = sorted({b + r for r in (0, 1, n // 2, n - 2, n - 1, 63, 64, 255, 256, 257) if 0 <= r < n})
    return rows


def _values(c, s, e):
    return oracle.mxfp4_dequantize(c[e].cpu().numpy(), s[e].cpu().numpy())


# one step of K, the ring's every residue, and loops of whole groups of steps
@pytest.mark.parametrize("nk,N,E,rows", [
    (1, 2048, 100, 20000), (2, 2048, 12, 32000), (3, 2048, 128, 24000), (4, 2048, 65, 20000), (5, 1536, 70, 30000),
    (6, 2048, 9, 20000), (8, 2048, 128, 20000), (9, 1024, 80, 40000), (11, 2816, 24, 30000),
])
@pytest.mark.parametrize("codes", [False, True])
def test_linear_many_tiles(moe, nk, N, E, rows, codes):
    K = 256 * nk
    rng = np.random.default_rng(nk * 1000 + E)
    sizes = _sizes(rng, E, rows)
    off, R = _offsets(sizes), sum(sizes)
    tiles = sum(-(-n // 256) for n in sizes) * (N // 256)
    print(f"mxfp4 linear of {tiles} tiles: K={K} N={N} E={E} R={R} codes={codes}", flush=True)
    assert tiles > 512 and R > 64 * E and -(-max(sizes) // 256) * (N // 256) <= 256
    g = torch.Generator(device="cuda").manual_seed(nk)
    c, s = _weights(moe, g, E, N, K, 0.02)
    x = _randn(g, R + TAIL, K)
    xf = host(x)
    xs = None
    if codes:
        x, xs = moe.mxfp4_quantize(x)
    y = torch.full((R + TAIL, N), 5.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_grouped_linear_mxfp4(x, c, s, torch.from_numpy(off).cuda(), x_scale=xs, out=y)
    assert torch.all(y[R:] == 5.0)
    for e in range(E):
        at, o, n = _one_expert(off, e)
        if n:
            one = moe.moe_grouped_linear_mxfp4(x[at], c[e:e + 1], s[e:e + 1], o, x_scale=None if xs is None else xs[at])
            assert torch.equal(one[:n], y[at][:n]), f"expert {e} of {n} rows"
    for e, at in _sample(off, rng).items():
        w = _values(c, s, e)[None]
        ref, mag = _product_ref(oracle.mxfp4_qdq(xf[at]), w, [0, len(at)])
        assert np.all(np.abs(host(y[at]) - ref) <= 2.0 ** -8 * np.abs(ref) + _steps(K) * mag + 1e-38), f"expert {e}"


# gate_up and down both of many tiles; H past seven steps reaches the whole groups of K steps
@pytest.mark.parametrize("H,I,E,rows", [
    (1536, 768, 100, 26000), (2048, 768, 128, 26000), (2304, 512, 70, 42000), (2816, 768, 40, 32000), (768, 1536, 66, 52000),
    (1280, 1024, 16, 33000),
])
@pytest.mark.parametrize("codes", [False, True])
def test_mlp_many_tiles(moe, H, I, E, rows, codes):
    rng = np.random.default_rng(H + I + E)
    sizes = _sizes(rng, E, rows)
    off, R = _offsets(sizes), sum(sizes)
    row_tiles = sum(-(-n // 256) for n in sizes)
    print(f"mxfp4 mlp of {row_tiles * (I // 128)} and {row_tiles * (H // 256)} tiles: H={H} I={I} E={E} R={R} codes={codes}", flush=True)
    assert row_tiles * min(I // 128, H // 256) > 512 and R > 64 * E and -(-max(sizes) // 256) * max(I // 128, H // 256) <= 256
    g = torch.Generator(device="cuda").manual_seed(H)
    c1, s1 = _weights(moe, g, E, 2 * I, H, 0.05)
    c2, s2 = _weights(moe, g, E, H, I, 0.05)
    x, prob = _randn(g, R + TAIL, H), 0.05 + torch.rand(R + TAIL, generator=g, device="cuda")
    xf = host(x)
    xs = None
    if codes:
        x, xs = moe.mxfp4_quantize(x)

    def mlp(at, o, w, out=None):
        return moe.moe_grouped_mlp_fwd(x[at], c1[w], c2[w], o, prob[at], compute="mxfp4", out=out,
                                       x_perm_scale=None if xs is None else xs[at], w_gate_up_scale=s1[w], w_down_scale=s2[w])

    y = torch.full((R + TAIL, H), 5.0, dtype=torch.bfloat16, device="cuda")
    mlp(slice(0, R + TAIL), torch.from_numpy(off).cuda(), slice(0, E), y)
    assert torch.all(y[R:] == 5.0)
    for e in range(E):
        at, o, n = _one_expert(off, e)
        if n:
            assert torch.equal(mlp(at, o, slice(e, e + 1))[:n], y[at][:n]), f"expert {e} of {n} rows"
    for e, at in _sample(off, rng).items():
        ref, tol = _mlp_tolerance(xf[at], _values(c1, s1, e)[None], _values(c2, s2, e)[None], [0, len(at)],
                                  host(prob[at]).astype(np.float64))
        assert np.all(np.abs(host(y[at]) - ref) <= tol), f"expert {e}"


# 8 to 64 rows an expert on average: 64 rows at a time, two units of 256 weights in flight in each
# of four wavefronts; 5 to 17 units reach the second buffer and its reloads
@pytest.mark.parametrize("K,N,sizes", [
    (1280, 256, [40, 0, 65, 17]), (2048, 512, [40, 0, 65, 17]), (2304, 256, [64, 1, 63, 0]), (2816, 256, [9, 128, 0, 16]),
    (3328, 256, [33, 48, 0, 130]), (4352, 768, [20, 20, 20, 20]),
])
@pytest.mark.parametrize("codes", [False, True])
def test_linear_rows_deep(moe, K, N, sizes, codes):
    assert 8 * len(sizes) < sum(sizes) + 3 <= 64 * len(sizes)
    _linear(moe, K, N, sizes, codes)


@pytest.mark.parametrize("H,I,sizes", [
    (1280, 2048, [40, 0, 65, 17]), (2304, 1280, [64, 1, 63, 0]), (2816, 256, [9, 128, 0, 16]), (3328, 2304, [33, 48, 0, 130]),
])
@pytest.mark.parametrize("act,wt", [("bf16", "codes"), ("codes", "codes")])
def test_mlp_rows_deep(moe, H, I, sizes, act, wt):
    assert 8 * len(sizes) < sum(sizes) <= 64 * len(sizes)
    _mlp(moe, H, I, sizes, act, wt)
