"""Every way that a product of the bf16 grouped MLP over 8-bit checkpoints is launched, with many rows of each
tile, against the float64 oracle (tolerances: test_gpu_ckpt8): whole tiles alone, whole tiles with the last
round's split along K, and split tiles behind a launch that has no whole one. Which way a call took shows in the
workspace: partial tiles are written by split products alone."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev_bf16, host
from moe_inputs import bf16_bits_to_f32, f32_to_bf16_bits
from test_gpu_ckpt8 import Case, _backward_check, _forward_check

pytestmark = pytest.mark.gpu
TILE = 256 * 256 * 4          # bytes of a float32 partial tile
HEADER = 8192                 # bytes before them: what is split
MARK = 0x7F


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_expert_gemm_amd as g
    g.lib()
    return g


class Marked:
    """The module with a marked workspace in each call of the grouped MLP; .touched: partial tiles written by the last."""

    def __init__(self, moe, c):
        self.moe, self.c = moe, c

    def __getattr__(self, name):
        return getattr(self.moe, name)

    def _call(self, fn, op, act, *args, **kw):
        from grouped_expert_gemm_amd import _lib
        desc = _lib.MlpDesc(self.c.E, self.c.H, self.c.I, _lib.MOE_BF16, act, _lib.MOE_BF16, 0)
        need = self.moe.workspace_size(op, desc, self.c.R)
        ws = torch.full((need,), MARK, dtype=torch.uint8, device="cuda")
        r = fn(*args, workspace=ws, **kw)
        cus = torch.cuda.get_device_properties(0).multi_processor_count
        part = ws[need - cus * TILE:].view(cus, TILE)
        self.touched = int((part != MARK).any(1).sum())
        return r

    def moe_grouped_mlp_fwd_ckpt8(self, *args):
        from grouped_expert_gemm_amd import _lib
        return self._call(self.moe.moe_grouped_mlp_fwd_ckpt8, _lib.MOE_OP_MLP_FWD, _lib.MOE_BF16, *args)

    def moe_grouped_mlp_bwd_ckpt8(self, *args, **kw):
        from grouped_expert_gemm_amd import _lib
        act = _lib.MOE_MXFP8 if "x_scale" in kw else _lib.MOE_BF16
        return self._call(self.moe.moe_grouped_mlp_bwd_ckpt8, _lib.MOE_OP_MLP_BWD_CKPT8, act, *args, **kw)


RAGGED = [1, 33, 129, 255, 256, 257, 300, 511, 40, 513]   # 15 row tiles
# On 256 CUs. Partial tiles of a call: the largest of its products' (tiles of the last round x chunks).
CASES = [
    # no product split: gate_up and down gradient have K = 512 and too many tiles for one launch that lists all;
    # down and gate_up gradient fill more than half a round (75 row tiles x 2)
    ("whole tiles", RAGGED * 5, 512, 1024, 0, 0),
    # gate_up 16 x 34 tiles, 32 of them in 8 chunks; down gradient 16 x 17 tiles, 16 of them in 16
    # chunks; down and gate_up gradient: 48 tiles in 5
    ("whole tiles and split ones", [257, 300, 385, 511, 512, 289, 260, 400], 768, 4352, 256, 256),
    # 64 rows of 3 of 128 experts: a launch that could hold whole tiles and has none. gate_up 24 tiles in 10
    # chunks, down 9 in 16; down gradient 12 in 16, gate_up gradient 9 in 16
    ("idle experts", [0] * 20 + [30] + [0] * 50 + [33] + [0] * 55 + [1], 768, 1024, 240, 192),
    # one launch that lists every tile: gate_up 12 tiles in 16 chunks (down, K = 512, whole); down gradient 6 in
    # 16, gate_up gradient 15 in 16
    ("split tiles alone", [200, 256, 131], 1280, 512, 192, 240),
]


@pytest.mark.parametrize("name,counts,H,I,fwd,bwd", CASES, ids=[c[0].replace(" ", "_") for c in CASES])
def test_forward_and_backward(moe, name, counts, H, I, fwd, bwd):
    print(f"ckpt8 {name}: {sum(counts)} rows of {len(counts)} experts, H={H} I={I}", flush=True)
    c = Case(counts, H, I, seed=H + I, behind=5)
    m = Marked(moe, c)
    zc, zs = _forward_check(m, c)
    same_card = torch.cuda.get_device_properties(0).multi_processor_count == 256
    assert not same_card or m.touched == fwd, f"{m.touched} partial tiles of the forward"
    tc, ts = moe.mxfp8_quantize(c.tokens)
    xv = oracle.mxfp8_dequantize(host(tc), host(ts))[c.src.cpu().numpy()]
    got = m.moe_grouped_mlp_bwd_ckpt8(c.dy, tc, zc, zs, c.prob, c.w1, c.w2, c.offsets, x_scale=ts, src_token=c.src)
    assert not same_card or m.touched == bwd, f"{m.touched} partial tiles of the backward"
    _backward_check(moe, c, zc, zs, got, xv, name)


def _rows_at_every_border(R, H):
    """bf16 rows whose blocks hold what a quantiser may get wrong: halfway values of normal and of subnormal codes, a
    largest magnitude of exactly 1.75 * 2^n and the next one above, exponents near both ends of float32."""
    g = np.random.default_rng(R + H)
    n = R * H // 32
    x = np.empty((n, 32))
    for i in range(n):
        kind = i % 6
        e = int(g.integers(-110, 110))
        sign = g.choice([-1.0, 1.0], 32)
        if kind == 0:      # halfway between two normal codes: four significant bits and a fifth
            x[i] = sign * (2 * g.integers(8, 16, 32) + 1) / 16 * np.exp2(e + g.integers(-4, 1, 32))
        elif kind == 1:    # subnormal codes and halfway between them, beside a largest value of 256 2^e
            x[i] = sign * (2 * g.integers(0, 9, 32) + g.integers(0, 2, 32)) * np.exp2(e - 10.0)
            x[i, int(g.integers(0, 32))] = 256 * np.exp2(float(e))
        elif kind in (2, 3):  # the largest value at and just above 1.75 * 2^n
            x[i] = sign * g.uniform(0, 1.7, 32) * np.exp2(float(e))
            x[i, int(g.integers(0, 32))] = (1.75 if kind == 2 else 1.7578125) * np.exp2(float(e))
        elif kind == 4:    # the smallest normal numbers: scale bytes from 0
            x[i] = sign * g.uniform(1, 2, 32) * np.exp2(g.integers(-126, -112, 32).astype(float))
        else:              # near the largest
            x[i] = sign * g.uniform(0, 1.9, 32) * np.exp2(g.integers(100, 128, 32).astype(float))
    x[x == 0] = 0.0        # no zero with a sign: a sum of products has none
    bits = f32_to_bf16_bits(x.reshape(R, H).astype(np.float32))
    return bf16_bits_to_f32(bits).astype(np.float64), dev_bf16(bits)


@pytest.mark.parametrize("counts", [[40], [300, 20], [1] * 129 + [70]], ids=["joined", "joined_two_row_tiles", "whole_tiles"])
def test_codes_of_exact_values(moe, counts):
    """W1 the identity: z is x itself, so codes and scales have one right answer."""
    print(f"ckpt8 exact codes {sum(counts)} rows of {len(counts)} experts", flush=True)
    c = Case(counts, 512, 256, seed=61)
    c.w1 = torch.eye(512, dtype=torch.bfloat16, device="cuda").repeat(c.E, 1, 1)
    x, c.x = _rows_at_every_border(c.R, 512)
    m = Marked(moe, c)
    _, zc, zs = m.moe_grouped_mlp_fwd_ckpt8(c.x, c.w1, c.w2, c.offsets, c.prob)
    assert (m.touched > 0) == (len(counts) < 100)
    codes, scales = oracle.mxfp8_quantize(x)
    assert np.array_equal(host(zs), scales), "scales"
    assert np.array_equal(host(zc), codes), "codes"
