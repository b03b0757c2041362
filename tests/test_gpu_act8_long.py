"""Tensors of more than 2^31 elements through the operators that hold activations in 8 bits: the last rows
lie past what a 32-bit index reaches. They are compared with the same rows in a call of their own."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_expert_gemm_amd as g
    g.lib()
    yield g
    torch.cuda.empty_cache()


def _tail(full, rows):
    """zeros of full's shape whose last rows are random; (tensor, those rows)"""
    t = torch.zeros(full, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(full[0])
    t[-rows:] = torch.randn((rows, full[1]), generator=g, device="cuda").to(torch.bfloat16)
    return t, t[-rows:].clone()


@pytest.mark.parametrize("H", [16384, 96])
def test_norm_and_read(moe, H):
    T, n = (1 << 31) // H + 40, 24
    print(f"add norm mxfp8 and read of {T} x {H}", flush=True)
    x, xs = _tail((T, H), n)
    w = torch.linspace(0.5, 1.5, H, device="cuda").to(torch.bfloat16)
    rows = torch.arange(T, device="cuda", dtype=torch.int32)
    r = moe.moe_add_norm_mxfp8(x, w, residual=x, row_id_map=rows, with_y=True, save_for_bwd=True)
    s = moe.moe_add_norm_mxfp8(xs, w, residual=xs, with_y=True, save_for_bwd=True)
    for name in ("sum", "y", "rstd", "codes", "scales"):
        assert torch.equal(r[name][-n:], s[name]), name
    assert not r["codes"][:8].any() and not r["sum"][:8].any()
    codes, scales, small, ss = r["codes"], r["scales"], s["codes"], s["scales"]
    del r, x
    v = moe.mxfp8_dequantize(codes, scales)
    assert torch.equal(v[-n:], moe.mxfp8_dequantize(small, ss)) and not v[:8].any()
    v = moe.mxfp8_dequantize(codes, scales, src_row=rows.flip(0), out=v)
    assert torch.equal(v[:n], moe.mxfp8_dequantize(small, ss).flip(0)) and not v[n:n + 8].any()


def test_forward_and_backward(moe):
    """The gate_up output past 2^31 elements (dZ past 2^32 bytes). n rows fill enough of a launch's last round
    that no gate_up tile is split along K in either call, so those sums run in one order; the products
    by H columns are few tiles and may be split, so they are compared within a few roundings."""
    H, I, n = 256, 14336, 300
    R = (1 << 31) // (2 * I) + 2 * n
    tiles = lambda rows: -(-rows // 256)
    while not ((tiles(R - n) + tiles(n)) * (I // 128)) % 256 > 128:
        R += 1
    print(f"ckpt8 of {R} rows, {2 * I} columns", flush=True)
    g = torch.Generator(device="cuda").manual_seed(2)
    w1 = (0.06 * torch.randn((2, 2 * I, H), generator=g, device="cuda")).bfloat16()
    w2 = (0.01 * torch.randn((2, H, I), generator=g, device="cuda")).bfloat16()
    x, xs = _tail((R, H), n)
    dy, dys = _tail((R, H), n)
    prob = torch.rand(R, generator=g, device="cuda")
    off = torch.tensor([0, R - n, R], dtype=torch.int32, device="cuda")
    offs = torch.tensor([0, 0, n], dtype=torch.int32, device="cuda")
    y, zc, zs = moe.moe_grouped_mlp_fwd_ckpt8(x, w1, w2, off, prob)
    ys, zcs, zss = moe.moe_grouped_mlp_fwd_ckpt8(xs, w1, w2, offs, prob[-n:].contiguous())
    assert torch.equal(zc[-n:], zcs) and torch.equal(zs[-n:], zss) and not zc[:300].any() and not zc[R - 2 * n:R - n].any()
    near = lambda a, b: float((a.float() - b.float()).norm()) <= 2.0 ** -8 * float(b.float().norm())
    assert near(y[-n:], ys) and not y[:300].any()
    xc, xsc = moe.mxfp8_quantize(x)
    xcs, xscs = moe.mxfp8_quantize(xs)
    src = torch.arange(R, device="cuda", dtype=torch.int32)
    dx, dw1, dw2, dprob = moe.moe_grouped_mlp_bwd_ckpt8(dy, xc, zc, zs, prob, w1, w2, off, x_scale=xsc, src_token=src)
    dxs, dw1s, dw2s, dprobs = moe.moe_grouped_mlp_bwd_ckpt8(dys, xcs, zcs, zss, prob[-n:].contiguous(), w1, w2, offs, x_scale=xscs)
    assert torch.equal(dprob[-n:], dprobs) and not dprob[:300].any()
    assert torch.equal(dw1[1], dw1s[1]) and torch.equal(dw2[1], dw2s[1]) and not dw1[0].any() and not dw2[0].any()
    assert near(dx[-n:], dxs) and not dx[:300].any()
