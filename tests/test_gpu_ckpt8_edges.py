"""Calls of the bf16 grouped MLP over 8-bit checkpoints at the edges of what its documentation allows."""
import pytest
import torch

from gpu_util import host
from test_gpu_ckpt8 import Case, _backward_check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_expert_gemm_amd as g
    g.lib()
    return g


def _dirty(moe, c, act):
    """A workspace whose every byte is 255 (a NaN in each type), so that what is read before it is written shows."""
    from grouped_expert_gemm_amd import _lib
    need = moe.workspace_size(_lib.MOE_OP_MLP_BWD_CKPT8, _lib.MlpDesc(c.E, c.H, c.I, _lib.MOE_BF16, act, _lib.MOE_BF16, 0), c.R)
    return torch.full((need,), 255, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("bad,good", [
    ([0, 130, 100], [0, 130, 130]), ([0, 40, 20, 150, -3], [0, 40, 40, 150, 150]), ([0, 9, 7, 5000], [0, 9, 9, 170]),
    ([0] + [2 * i for i in range(1, 71)] + [30] * 60, [0] + [2 * i for i in range(1, 71)] + [140] * 60)])
def test_offsets_that_decrease_are_read_as_their_running_maximum(moe, bad, good):
    """By every part of the backward alike: the gradients are those of the repaired offsets, bit for bit."""
    from grouped_expert_gemm_amd import _lib
    print(f"ckpt8 offsets {bad[:6]}", flush=True)
    c = Case([0] * (len(good) - 1), 256, 256, seed=12, behind=170)
    offs = [torch.tensor(o, dtype=torch.int32, device="cuda") for o in (good, bad)]
    _, zc, zs = moe.moe_grouped_mlp_fwd_ckpt8(c.x, c.w1, c.w2, offs[0], c.prob)
    tc, ts = moe.mxfp8_quantize(c.tokens)
    rc, rs = tc[c.src.long()].contiguous(), ts[c.src.long()].contiguous()
    n = good[-1]
    for kw in (dict(x=tc, x_scale=ts, src_token=c.src), dict(x=rc, x_scale=rs), dict(x=moe.mxfp8_dequantize(rc, rs))):
        act = _lib.MOE_BF16 if "x_scale" not in kw else _lib.MOE_MXFP8
        got = []
        for o in offs:
            dx = torch.full_like(c.dy, 5.0)
            r = moe.moe_grouped_mlp_bwd_ckpt8(c.dy, kw["x"], zc, zs, c.prob, c.w1, c.w2, o, x_scale=kw.get("x_scale"),
                                              src_token=kw.get("src_token"), dx_perm=dx, workspace=_dirty(moe, c, act))
            assert bool((dx[n:] == 5.0).all())
            got.append((dx, r[1], r[2], r[3][:n]))
        for a, b, name in zip(*got, ("dx", "dw1", "dw2", "dprob")):
            assert torch.equal(a, b), name
            assert not bool(torch.isnan(a.float()).any()), name


@pytest.mark.parametrize("counts", [[40, 0, 9], [1] * 129 + [5]])
def test_slope_of_the_gate_at_any_magnitude(moe, counts):
    """Gates from 2^-36 to 2^52 on both sides: silu' = sig + g sig (1 - sig) goes to 1 above (where float32's 1 beside
    g vanishes from 2^24 on) and to 0 below. W1 is the identity, so that dx is dZ itself, each column apart. The
    second case's tiles are too many to be split along K: the down gradient's own epilogue, else the join's."""
    print(f"ckpt8 gates of any magnitude {len(counts)} experts", flush=True)
    c = Case(counts, 512, 256, seed=51)
    c.w1 = torch.eye(512, dtype=torch.bfloat16, device="cuda").repeat(c.E, 1, 1)
    g = torch.Generator(device="cuda").manual_seed(52)
    zc = torch.randint(0, 127, (c.R, 512), generator=g, device="cuda") + 128 * torch.randint(0, 2, (c.R, 512), generator=g, device="cuda")
    zs = torch.randint(100, 171, (c.R, 16), generator=g, device="cuda")
    zs[:, 8:] = torch.randint(118, 128, (c.R, 8), generator=g, device="cuda")
    zc, zs = zc.to(torch.uint8), zs.to(torch.uint8)
    got = moe.moe_grouped_mlp_bwd_ckpt8(c.dy, c.x, zc, zs, c.prob, c.w1, c.w2, c.offsets)
    _backward_check(moe, c, zc, zs, got, host(c.x), "gates of any magnitude")


def test_no_kept_token(moe):
    """T = 0: every token is out of [0, T) and read as zeros, x has no row and may be NULL."""
    c = Case([30, 0, 9], 256, 256, seed=14)
    _, zc, zs = moe.moe_grouped_mlp_fwd_ckpt8(c.x, c.w1, c.w2, c.offsets, c.prob)
    none = torch.zeros((0, 256), dtype=torch.uint8, device="cuda")
    got = moe.moe_grouped_mlp_bwd_ckpt8(c.dy, none, zc, zs, c.prob, c.w1, c.w2, c.offsets, x_scale=none.view(0, 256)[:, :8].contiguous(),
                                        src_token=c.src)
    want = moe.moe_grouped_mlp_bwd_ckpt8(c.dy, torch.zeros_like(c.x), zc, zs, c.prob, c.w1, c.w2, c.offsets)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and not got[1].any() and bool(got[2].any())
