"""Which codes moe_permute takes a uint8 tensor for, by the scales that come with it: MXFP8 where
they are a byte per 32 bytes of x (in any shape), MXFP4 where they are [T, bytes of a row / 16], and
a refusal where there are fewer than the rows need. The binding's call is recorded on the CPU;
nothing is launched."""
import pytest
import torch

import grouped_expert_gemm_amd as moe
from grouped_expert_gemm_amd import MOE_MXFP4, MOE_MXFP8


@pytest.fixture
def calls(monkeypatch):
    seen = []

    class Lib:
        def moe_permute(self, x, x_scale, dt, T, H, E, k, *rest):
            seen.append((dt, T, H, k))
            return 0

    monkeypatch.setattr(moe, "lib", lambda: Lib())
    monkeypatch.setattr(moe, "_need_cuda", lambda *ts: None)
    monkeypatch.setattr(moe, "_stream", lambda device=None: None)
    monkeypatch.setattr(moe, "workspace_size", lambda *a: 16)
    return seen


def _permute(T, row_bytes, scale, k=2):
    x = torch.zeros((T, row_bytes), dtype=torch.uint8)
    idx = torch.zeros((T, k), dtype=torch.int32)
    return moe.moe_permute(x, idx, None, 4, x_scale=scale)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 64])
def test_which_codes(calls, T):
    u8 = lambda *shape: torch.zeros(shape, dtype=torch.uint8)  # noqa: E731
    r = _permute(T, 256, u8(T, 8))
    assert calls[-1] == (MOE_MXFP8, T, 256, 2) and r["x_perm_scale"].shape == (2 * T, 8)
    # the same scales as one run of bytes: for two tokens as many as a row of MXFP4 scales has
    r = _permute(T, 256, u8(T * 8))
    assert calls[-1] == (MOE_MXFP8, T, 256, 2) and r["x_perm_scale"].shape == (2 * T, 8)
    r = _permute(T, 256, u8(1, T * 8))
    assert calls[-1] == (MOE_MXFP8, T, 256, 2)
    r = _permute(T, 256, u8(T, 16))
    assert calls[-1] == (MOE_MXFP4, T, 512, 2) and r["x_perm"].shape == (2 * T, 256)
    assert r["x_perm_scale"].shape == (2 * T, 16)


def test_too_few_scales_are_refused(calls):
    for T, n in ((4, (4, 7)), (4, (3, 8)), (4, (1, 16)), (2, (15,)), (64, (16, 16))):
        with pytest.raises(ValueError):
            _permute(T, 256, torch.zeros(n, dtype=torch.uint8))
    assert not calls
    with pytest.raises(ValueError):   # the reused map gathers the same scales
        moe.moe_permute(torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.int32), None, 4,
                        x_scale=torch.zeros((3, 8), dtype=torch.uint8), row_id_map=torch.zeros(8, dtype=torch.int32))
    assert not calls


@pytest.mark.gpu
def test_two_tokens_with_their_scales_in_one_run():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print("permute of two tokens, flat MXFP8 scales", flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((2, 256), generator=g, device="cuda").to(torch.bfloat16)
    idx = torch.tensor([[1, 3], [0, 1]], dtype=torch.int32, device="cuda")
    c, s = moe.mxfp8_quantize(x)
    a = moe.moe_permute(c, idx, None, 4, x_scale=s)
    b = moe.moe_permute(c, idx, None, 4, x_scale=s.view(-1))
    assert torch.equal(a["x_perm"], b["x_perm"]) and torch.equal(a["x_perm_scale"], b["x_perm_scale"])
    want = s[a["src_token"].long()]
    assert torch.equal(b["x_perm_scale"], want)
