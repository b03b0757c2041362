"""Reading MXFP8 rows by index where an index names no row: zeros in a new tensor, untouched rows in a given one."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_expert_gemm_amd as g
    g.lib()
    return g


@pytest.mark.parametrize("rows,cols,n", [(1, 32, 5), (7, 96, 300), (64, 1440, 1000), (0, 64, 9)])
def test_missing_rows(moe, rows, cols, n):
    print(f"read mxfp8 {rows} x {cols} to {n} rows", flush=True)
    g = torch.Generator(device="cuda").manual_seed(n)
    codes = torch.randint(0, 127, (rows, cols), generator=g, device="cuda").to(torch.uint8)
    scales = torch.randint(90, 160, (rows, cols // 32), generator=g, device="cuda").to(torch.uint8)
    src = torch.randint(-2, rows + 3, (n,), generator=g, device="cuda").int()
    src[0], src[-1] = -2 ** 31, 2 ** 31 - 1
    lost = (src < 0) | (src >= rows)
    full = torch.zeros((n, cols), dtype=torch.bfloat16, device="cuda")
    full[~lost] = moe.mxfp8_dequantize(codes, scales)[src[~lost].long()]
    for _ in range(3):
        held = torch.full((n, cols), float("nan"), dtype=torch.bfloat16, device="cuda")
        del held                                    # the allocator hands this memory out again
        assert torch.equal(moe.mxfp8_dequantize(codes, scales, src_row=src), full)
    out = torch.full((n, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    full[lost] = 7.0
    assert torch.equal(moe.mxfp8_dequantize(codes, scales, src_row=src, out=out), full)


def test_missing_rows_in_a_graph(moe):
    codes = torch.randint(0, 127, (50, 256), device="cuda").to(torch.uint8)
    scales = torch.full((50, 8), 127, dtype=torch.uint8, device="cuda")
    src = torch.arange(-20, 80, device="cuda").int()
    moe.mxfp8_dequantize(codes, scales, src_row=src)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = moe.mxfp8_dequantize(codes, scales, src_row=src)
    for _ in range(4):
        src.copy_(torch.randint(-5, 55, (100,), device="cuda"))
        out.fill_(float("nan"))
        graph.replay()
        assert torch.equal(out, moe.mxfp8_dequantize(codes, scales, src_row=src)) and not bool(out[(src < 0) | (src > 49)].any())


def test_refusals(moe):
    c = torch.zeros((4, 64), dtype=torch.uint8, device="cuda")
    s = torch.zeros((4, 2), dtype=torch.uint8, device="cuda")
    m = torch.zeros(4, dtype=torch.int32, device="cuda")
    for kw in (dict(src_row=m.long()), dict(src_row=m.view(2, 2)), dict(scales=s[:3].contiguous()), dict(codes=c.int())):
        with pytest.raises(ValueError, match="mxfp8_dequantize"):
            moe.mxfp8_dequantize(**{"codes": c, "scales": s, "src_row": m, **kw})
    with pytest.raises(moe.MoeError, match="cols % 32"):
        moe.mxfp8_dequantize(c[:, :48].contiguous(), s[:, :1].contiguous(), src_row=m)
