"""The gate's gradient of the bf16 grouped MLP's backward at gates of any magnitude, against the float64 oracle."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import host

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = 2.0 ** -8


def test_slope_of_the_gate_at_any_magnitude():
    """silu' = sig + g sig (1 - sig) is 1 for large gates (float32's 1 beside g vanishes from 2^24 on). W1 is the
    identity, so that dx is dZ itself. Tolerance: dH's float32 sum of H products (H u of their magnitudes), 20 u for
    exponential, reciprocal and products against the sum of the slope's magnitudes, and one rounding to bf16; a
    second one changes nothing (dZ's values pass the product with the identity as they are)."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_expert_gemm_amd as moe
    H, I, E, R = 512, 256, 3, 150
    g = torch.Generator(device="cuda").manual_seed(8)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    off = np.array([0, 60, 60, R])
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    w1 = torch.eye(H, dtype=torch.bfloat16, device="cuda").repeat(E, 1, 1)
    w2, x, dy = (I ** -0.5 * n(E, H, I)).bfloat16(), n(R, H).bfloat16(), n(R, H).bfloat16()
    gates = n(R, I) * torch.exp2(torch.randint(-36, 53, (R, I), generator=g, device="cuda").float())
    z = torch.cat([gates, n(R, I)], 1).bfloat16()
    prob = torch.rand(R, generator=g, device="cuda") + 0.1
    h = torch.zeros((R, I), dtype=torch.bfloat16, device="cuda")
    dx = host(moe.moe_grouped_mlp_bwd(dy, x, z, h, prob, w1, w2, offsets)[0])
    zf, p = host(z), host(prob).astype(np.float64)[:, None]
    ref = oracle.grouped_mlp_backward_from_z(host(dy), host(x), zf, host(w1), host(w2), off, p[:, 0])["dz"]
    gf, u = zf[:, :I], zf[:, I:]
    sig = 1 / (1 + np.exp(-np.clip(gf, -700, None)))
    for e in (0, 2):
        r = slice(off[e], off[e + 1])
        dh, mag = np.abs(host(dy)[r] @ host(w2)[e]), np.abs(host(dy)[r]) @ np.abs(host(w2)[e])
        err = H * U * mag + 20 * U * dh
        tol = np.concatenate([err * np.abs(p[r] * u[r]) * (sig[r] + np.abs(gf[r]) * sig[r] * (1 - sig[r])),
                              err * np.abs(p[r] * gf[r]) * sig[r]], 1)
        q = np.abs(dx[r] - ref[r]) / (HALF * np.abs(ref[r]) + (1 + HALF) * tol + 1e-30)
        assert np.all(q <= 1), f"dZ of expert {e}: {q.max():.2f} times the tolerance"
