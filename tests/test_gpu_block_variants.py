"""Kernel variants that calls of realistic size take: norms of at least 1024 rows that one wavefront
holds in four vectors a lane (whole vectors and not, over one and over several rows a wavefront), and
balance losses of runs long enough for four tokens in flight, in one and several sequences.
Tolerances and checks are those of test_gpu_norm.py and test_gpu_balance.py; at T = 9000 and H >= 1032 a
column sum of the backward adds runs of 5 tokens, 29 of 1800 partial sums in each of 64 threads, and
those: 5 + 29 + 18 + 4 roundings, within the 128 taken there."""
import numpy as np
import pytest
import torch

from test_gpu_balance import _check, _inputs
from test_gpu_norm import Maker, _post
from test_gpu_norm import test_pre_norm as _pre

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_expert_gemm_amd as g
    g.lib()
    return g


# 129 to 256 vectors of 8 bf16 or 4 float32 a row
@pytest.mark.parametrize("dtype,T,H,k,kind,group,scale,next_norm", [
    ("bf16", 1100, 1032, 1, "none", 1, 1.0, True),
    ("bf16", 1100, 1032, 8, "channel", 300, 0.5, False),
    ("bf16", 1100, 1999, 8, "token", 1, 1.0, True),
    ("bf16", 1025, 1999, 1, "channel", 1025, 1.0, False),
    ("bf16", 1300, 2048, 8, "token", 1, 1.0, True),
    ("bf16", 1101, 2048, 3, "none", 1, -1.0, False),
    ("bf16", 9000, 1032, 1, "channel", 64, 1.0, True),
    ("f32", 1100, 516, 1, "none", 1, 1.0, True),
    ("f32", 1100, 1001, 8, "token", 1, 1.0, True),
    ("f32", 1101, 1001, 1, "channel", 250, 2.0, False),
    ("f32", 1100, 1024, 8, "channel", 275, 1.0, True),
    ("f32", 1300, 1024, 1, "none", 1, 1.0, False),
])
def test_post_norm(moe, dtype, T, H, k, kind, group, scale, next_norm):
    print(f"post norm of many rows {dtype} T={T} H={H} k={k} gate={kind}/{group}", flush=True)
    _post(moe, Maker(T * 31 + H, dtype), T, H, k, kind, group, scale, next_norm)


@pytest.mark.parametrize("dtype,T,H", [("bf16", 1100, 1032), ("bf16", 1025, 1999), ("bf16", 9000, 2048), ("f32", 1100, 513),
                                       ("f32", 1101, 1001), ("f32", 9001, 1024)])
def test_pre_norm(moe, dtype, T, H):
    _pre(moe, dtype, T, H)


# runs of more than 2048 lanes' worth of tokens, in more than one workgroup a sequence; 64, 32 and 16
# lanes a token; whole 16-byte rows and not; last runs that are no multiple of the tokens in flight
@pytest.mark.parametrize("S,L,E,k", [(1, 33001, 256, 8), (1, 70001, 256, 8), (1, 50003, 255, 6), (1, 70013, 128, 8),
                                     (1, 140001, 37, 2), (3, 40007, 256, 4), (4, 20011, 130, 3)])
def test_balance_long_runs(moe, S, L, E, k):
    T = S * L
    rng, logits, idx = _inputs(T + E, T, E, k)
    _check(moe, logits, idx, 0.01, 0.001, L, None, None, None, "long runs")
    mask = (np.arange(L)[None] < rng.integers(L // 3, L + 1, (S, 1))).astype(np.uint8).ravel()
    mask[rng.integers(0, T, T // 50)] = 0
    d_in = (1e-4 * rng.standard_normal((T, E))).astype(np.float32)
    _check(moe, logits, idx, 1.0, 0.5, L, mask, np.array([-1.75], np.float32), d_in, "long runs, padded")
