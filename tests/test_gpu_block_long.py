"""Tensors of more than 2^31 elements through the block's operators: the last rows lie past what a
32-bit index reaches. They are compared, bit for bit or within what a different order of sums can
change, with the same rows in a call of their own."""
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


@pytest.mark.parametrize("H", [16384, 16383])
def test_norms(moe, H):
    T, n = (1 << 31) // H + 40, 24
    print(f"norms of {T} x {H}", flush=True)
    x, xs = _tail((T, H), n)
    w = torch.linspace(0.5, 1.5, H, device="cuda").to(torch.bfloat16)
    y, r = moe.moe_pre_norm(x, w, save_rstd=True)
    ys, rs = moe.moe_pre_norm(xs, w, save_rstd=True)
    assert torch.equal(y[-n:], ys) and torch.equal(r[-n:], rs) and not y[:8].any()
    rows = torch.arange(T, device="cuda", dtype=torch.int32)
    o = moe.moe_post_norm(y, x, w, row_id_map=rows, save_for_bwd=True)
    os_ = moe.moe_post_norm(ys, xs, w, save_for_bwd=True)
    for name in ("out", "c", "rstd"):
        assert torch.equal(o[name][-n:], os_[name]), name
    del y
    b = moe.moe_post_norm_bwd(x, o["c"], o["rstd"], w, row_id_map=rows)
    bs = moe.moe_post_norm_bwd(xs, os_["c"], os_["rstd"], w)
    assert torch.equal(b["dy"][-n:], bs["dy"]) and not b["dy"][:8].any()
    # all other rows add zeros, so both are sums of the same n terms, each off by at most n half steps
    err = (b["dweight"].double() - bs["dweight"].double()).abs()
    mag = (xs.double() * os_["c"].double() * os_["rstd"].double()[:, None]).abs().sum(0)
    assert (err <= 2 * n * 2.0 ** -24 * mag + 1e-30).all()
    dx, _ = moe.moe_pre_norm_bwd(b["dy"], x, w, r)
    dxs, _ = moe.moe_pre_norm_bwd(bs["dy"], xs, w, rs)
    assert torch.equal(dx[-n:], dxs)


def test_balance_loss(moe):
    E, k, n = 256, 2, 64
    T = (1 << 31) // E + 4 * n
    T -= T % n
    print(f"balance loss of {T} x {E}", flush=True)
    logits = torch.zeros((T, E), device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    logits[-n:] = torch.randn((n, E), generator=g, device="cuda")
    idx = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    idx[-n:] = moe.moe_route_topk(logits[-n:].contiguous(), k)[0]
    mask = torch.zeros(T, dtype=torch.bool, device="cuda")
    mask[-n:] = True   # only the last sequence counts
    loss, counts, tokens = moe.moe_balance_loss(logits, idx, 1.0, 0.5, seq_len=n, mask=mask)
    ls, cs, ts = moe.moe_balance_loss(logits[-n:].contiguous(), idx[-n:].contiguous(), 1.0, 0.5)
    assert torch.equal(counts[-1:], cs) and int(counts[:-1].abs().max()) == 0
    assert int(tokens[-1]) == 1 and int(tokens[-2]) == n and int(ts[0]) == n
    # the same sums in another order: 64 terms and 256, 2^-24 of their size each
    assert torch.allclose(loss, ls, rtol=400 * 2.0 ** -24, atol=0)
    d = moe.moe_balance_loss_bwd(logits, counts, tokens, k, 1.0, 0.5, seq_len=n, mask=mask)
    ds = moe.moe_balance_loss_bwd(logits[-n:].contiguous(), cs, ts, k, 1.0, 0.5)
    assert torch.equal(d[-n:], ds) and not d[:n].any()


@pytest.mark.parametrize("codes", [False, True])
def test_mxfp4_linear(moe, codes):
    """Outputs past 2^31 elements and 2^32 bytes (256-row tiles)."""
    K, N, n = 256, 8192, 300
    R = (1 << 31) // N + 2 * n
    print(f"mxfp4 linear of {R} x {N}, codes={codes}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randn((2 * N, K), generator=g, device="cuda").to(torch.bfloat16)
    wc, ws = moe.mxfp4_quantize(w)
    wc, ws = wc.view(2, N, K // 2), ws.view(2, N, K // 32)
    x, xs = _tail((R, K), n)
    off = torch.tensor([0, R - n, R], dtype=torch.int32, device="cuda")
    offs = torch.tensor([0, 0, n], dtype=torch.int32, device="cuda")
    if codes:
        c, s = moe.mxfp4_quantize(x)
        y = moe.moe_grouped_linear_mxfp4(c, wc, ws, off, x_scale=s)
    else:
        y = moe.moe_grouped_linear_mxfp4(x, wc, ws, off)
    ys = moe.moe_grouped_linear_mxfp4(xs, wc, ws, offs)
    assert torch.equal(y[-n:], ys) and not y[:300].any() and not y[R - 2 * n:R - n].any()


def test_mxfp4_quantise(moe):
    cols, n = 8192, 16
    rows = (1 << 32) // cols + 64   # codes past 2^31 bytes
    print(f"mxfp4 quantise {rows} x {cols}", flush=True)
    x, xs = _tail((rows, cols), n)
    c, s = moe.mxfp4_quantize(x)
    cs, ss = moe.mxfp4_quantize(xs)
    assert torch.equal(c[-n:], cs) and torch.equal(s[-n:], ss) and not c[:n].any()
    del x
    v = moe.mxfp4_dequantize(c, s)
    assert torch.equal(v[-n:], moe.mxfp4_dequantize(cs, ss)) and not v[:n].any()
