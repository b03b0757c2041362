"""One MoE block whose activations are held in 8 bits, as a model's layer runs it. Training: residual
add + norm (codes kept) -> router -> permute -> experts (gate_up output kept in MXFP8) -> combine +
residual + the next norm, and the whole backward from what was kept. Serving: the same norms feeding
MXFP8 experts.

Training is compared with the float64 oracle on the values that were kept, then captured into a graph
and replayed, run on two streams at once, and two captured calls share a workspace.

End to end (bf16, float32 sums): each bf16 tensor on the way rounds by at most 2^-8 of its value and the
roundings of different elements are independent, so the relative error of a gradient tensor's norm
stays below the sum over the roundings on its path (at most 10 tensors) of 2^-8: 4e-2."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from gpu_util import host

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_expert_gemm_amd as g
    g.lib()
    return g


class Layer:
    def __init__(self, seed, H, I, E):
        g = torch.Generator(device="cuda").manual_seed(seed)
        bf = lambda *s, scale=1.0, mean=0.0: (mean + scale * torch.randn(s, generator=g, device="cuda")).to(torch.bfloat16)
        self.H, self.I, self.E = H, I, E
        self.wn1, self.wn2 = (bf(H, scale=0.1, mean=1.0) for _ in range(2))
        self.wr = bf(E, H, scale=H ** -0.5)
        self.w1, self.w2 = bf(E, 2 * I, H, scale=H ** -0.5), bf(E, H, I, scale=I ** -0.5)


def _inputs(seed, T, H):
    """The residual stream, the attention's output, the gradients of the next norm's output and of the stream."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16) for _ in range(4)]


def _step(moe, p, inp, k):
    x, attn, du, dstream = inp
    T = x.shape[0]
    a = moe.moe_add_norm_mxfp8(attn, p.wn1, residual=x, eps=EPS, with_y=True, save_for_bwd=True)
    logits = moe.moe_router_logits(a["y"], p.wr)
    idx, prob = moe.moe_route_topk(logits, k)
    m = moe.moe_permute(a["y"], idx, prob, p.E)
    y, zc, zs = moe.moe_grouped_mlp_fwd_ckpt8(m["x_perm"], p.w1, p.w2, m["offsets"], m["prob_perm"])
    b = moe.moe_add_norm_mxfp8(y, p.wn2, residual=a["sum"], row_id_map=m["row_id_map"], k=k, eps=EPS, with_y=True,
                               save_for_bwd=True)
    # backward
    ds, dwn2 = moe.moe_pre_norm_bwd(du, b["sum"], p.wn2, b["rstd"], dx_in=dstream)
    dyp = moe.moe_permute(ds, idx, None, p.E, row_id_map=m["row_id_map"])["x_perm"]
    dxp, dw1, dw2, dprob = moe.moe_grouped_mlp_bwd_ckpt8(dyp, a["codes"], zc, zs, m["prob_perm"], p.w1, p.w2, m["offsets"],
                                                         x_scale=a["scales"], src_token=m["src_token"])
    da = moe.moe_unpermute_combine(dxp, m["row_id_map"], T, k)
    dp = torch.index_select(dprob, 0, m["row_id_map"].long()).view(T, k)
    dl = moe.moe_route_topk_bwd(idx, prob, dp, p.E)
    da, dwr = moe.moe_router_bwd(a["y"], p.wr, dl, dx_in=da)
    dx, dwn1 = moe.moe_pre_norm_bwd(da, a["sum"], p.wn1, a["rstd"], dx_in=ds)
    fwd = dict(a=a, b=b, idx=idx, m=m, zc=zc, zs=zs)
    return fwd, dict(dx=dx, dwn1=dwn1, dwn2=dwn2, dwr=dwr, dw1=dw1, dw2=dw2)


def _flat(f, g):
    return [*(f["a"][n] for n in ("sum", "y", "rstd", "codes", "scales")), *(f["b"][n] for n in ("sum", "y", "rstd", "codes", "scales")),
            f["zc"], f["zs"], *g.values()]


def _bytes(t):
    return t.contiguous().view(torch.uint8)


def _rel(got, ref):
    got = host(got).astype(np.float64)
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("T,H,I,E,k", [(96, 256, 256, 8, 2), (65, 512, 256, 16, 4), (1, 256, 256, 4, 1), (700, 256, 512, 4, 2)])
def test_training_step_against_the_oracle(moe, T, H, I, E, k):
    print(f"8-bit block training step T={T} H={H} I={I} E={E} k={k}", flush=True)
    p = Layer(T + H, H, I, E)
    inp = _inputs(T, T, H)
    f, g = _step(moe, p, inp, k)
    X, At, Du, Ds = (host(t) for t in inp)
    wn1, wn2, wr, w1, w2 = (host(t) for t in (p.wn1, p.wn2, p.wr, p.w1, p.w2))
    idx = host(f["idx"])
    s1 = X + At
    a, r1 = oracle.pre_norm(s1, wn1, EPS)
    assert _rel(f["a"]["y"], a) < 4e-2 and _rel(f["a"]["sum"], s1) < 4e-2
    lg = np.take_along_axis(a @ wr.T, idx, 1)
    e = np.exp(lg - lg.max(1, keepdims=True))
    prob = e / e.sum(1, keepdims=True)
    m = oracle.permute(idx, E)
    src, slot, rows = m["src_token"], m["src_slot"], np.asarray(m["row_id_map"]).reshape(T, k)
    pp = prob.ravel()[src * k + slot]
    y = oracle.grouped_mlp_forward(a[src], w1, w2, m["offsets"], pp)[0]
    s2 = oracle.add_rows(y, s1, rows)
    u, r2 = oracle.pre_norm(s2, wn2, EPS)
    assert _rel(f["b"]["y"], u) < 4e-2 and _rel(f["b"]["sum"], s2) < 4e-2
    # what was kept, as values: half a step of E4M3 is 2^-4 of a value at most
    kept_x = oracle.mxfp8_dequantize(host(f["a"]["codes"]), host(f["a"]["scales"]))
    kept_z = oracle.mxfp8_dequantize(host(f["zc"]), host(f["zs"]))
    z = np.concatenate([a[src[o:n]] @ w1[i].T for i, (o, n) in enumerate(zip(m["offsets"][:-1], m["offsets"][1:]))])
    assert np.linalg.norm(kept_x - a) <= 2.0 ** -4 * np.linalg.norm(a) and np.linalg.norm(kept_z - z) <= (2.0 ** -4 + 4e-2) * np.linalg.norm(z)
    ds, dwn2 = oracle.pre_norm_backward(Du, s2, wn2, r2, Ds)

    def backward(values_z, values_x):
        gb = oracle.grouped_mlp_backward_from_z(ds[src], values_x[src], values_z, w1, w2, m["offsets"], pp)
        da = np.zeros((T, H))
        np.add.at(da, src, gb["dx_perm"])
        dl = oracle.route_topk_backward(a @ wr.T, idx, gb["dprob_perm"][rows])
        da_r, dwr = oracle.router_backward(a, wr, dl)
        dx, dwn1 = oracle.pre_norm_backward(da + da_r, s1, wn1, r1, ds)
        return dict(dx=dx, dwn1=dwn1, dwn2=dwn2, dw1=gb["dw_gate_up"], dw2=gb["dw_down"], dwr=dwr)

    ref, exact = backward(kept_z, kept_x), backward(z, a)
    for n in ("dx", "dwn1", "dwn2", "dw1", "dw2") + (("dwr",) if k > 1 else ()):
        assert _rel(g[n], ref[n]) < 4e-2, n
    # What 8 bits cost against the unrounded backward: h = silu(G) U p moves by at most (1 + |G| (1 - sig) + 1) 2^-4
    # of itself (the bracket is below 2.3 for G > 0, and |G| (1 - sig) grows only where silu vanishes), x by 2^-4,
    # independently by element
    for n, bound in (("dw2", 2.3 / 16 + 4e-2), ("dw1", (2 * 2.3 + 1) / 16 + 4e-2), ("dx", 2 * 2.3 / 16 + 4e-2)):
        assert _rel(g[n], exact[n]) < bound, n


def test_graph_replays(moe):
    """Captured once, replayed on new inputs between eager runs, bit for bit the eager step."""
    T, H, I, E, k = 512, 512, 256, 16, 2
    print("8-bit block training step under graph capture", flush=True)
    p = Layer(3, H, I, E)
    buf = _inputs(100, T, H)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(moe, p, buf, k)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = _flat(*_step(moe, p, buf, k))
    for rep in range(4):
        new = _inputs(200 + rep, T, H)
        for dst, src in zip(buf, new):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in static]
        ref = _flat(*_step(moe, p, new, k))
        torch.cuda.synchronize()
        for i, (s, r) in enumerate(zip(got, ref)):
            assert torch.equal(_bytes(s), _bytes(r)), f"replay {rep}: tensor {i}"


def test_two_streams_at_once(moe):
    """Two blocks in flight on two streams, each with its own workspaces, equal the same calls alone."""
    T, H, I, E, k = 1024, 512, 256, 16, 2
    print("two 8-bit blocks on two streams", flush=True)
    p = Layer(5, H, I, E)
    ins = [_inputs(300 + i, T, H) for i in range(2)]
    ref = [_flat(*_step(moe, p, i, k)) for i in ins]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for rep in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = _flat(*_step(moe, p, ins[i], k))
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(got[i], ref[i]):
            assert torch.equal(_bytes(a), _bytes(b))


def test_two_graphs_share_a_workspace(moe):
    """Captured forwards and backwards of two sizes, replayed one after the other on one stream with one
    workspace between them, scribbled over in between."""
    H, I, E = 256, 512, 4
    print("two graphs, one workspace", flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    w1, w2 = n(E, 2 * I, H) * 0.06, n(E, H, I) * 0.04
    from grouped_expert_gemm_amd import _lib
    sizes = (40, 900)
    need = max(moe.workspace_size(op, _lib.MlpDesc(E, H, I, 1, act, 1, 0), R) for R in sizes
               for op, act in ((_lib.MOE_OP_MLP_FWD, 1), (_lib.MOE_OP_MLP_BWD_CKPT8, _lib.MOE_MXFP8)))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    calls, refs = [], []
    for R in sizes:
        x, dy, prob = n(R, H), n(R, H), torch.rand(R, generator=g, device="cuda")
        off = torch.linspace(0, R, E + 1, device="cuda").int()
        xc, xs = moe.mxfp8_quantize(x)

        def call(workspace=None, x=x, dy=dy, prob=prob, off=off, xc=xc, xs=xs):
            y, zc, zs = moe.moe_grouped_mlp_fwd_ckpt8(x, w1, w2, off, prob, workspace=workspace)
            return [y, zc, zs, *moe.moe_grouped_mlp_bwd_ckpt8(dy, xc, zc, zs, prob, w1, w2, off, x_scale=xs, workspace=workspace)]

        calls.append(call)
        refs.append(call())
    torch.cuda.synchronize()
    graphs, outs = [], []
    for call in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call(ws))
        graphs.append(graph)
    for rep in range(3):
        for i in (0, 1, 1, 0):
            for t in outs[i]:
                t.zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            for a, b in zip(outs[i], refs[i]):
                assert torch.equal(_bytes(a), _bytes(b)), f"replay {rep} of graph {i}"
            ws.fill_(0xA5)


def _serve(moe, p, x, y_in, q, k):
    a = moe.moe_add_norm_mxfp8(y_in, p.wn1, residual=x, eps=EPS, with_y=True)
    idx, prob = moe.moe_route_topk(moe.moe_router_logits(a["y"], p.wr), k)
    m = moe.moe_permute(a["codes"], idx, prob, p.E, x_scale=a["scales"])
    y = moe.moe_grouped_mlp_fwd(m["x_perm"], q[0], q[2], m["offsets"], m["prob_perm"], compute="mxfp8",
                                x_perm_scale=m["x_perm_scale"], w_gate_up_scale=q[1], w_down_scale=q[3])
    b = moe.moe_add_norm_mxfp8(y, p.wn2, residual=a["sum"], row_id_map=m["row_id_map"], k=k, eps=EPS, with_y=True)
    return a, b, idx, prob, m


@pytest.mark.parametrize("T", [1, 7, 300])
def test_serving_step(moe, T):
    """MXFP8 experts fed by the norm's codes, against the oracle on those codes (the MXFP8 path's own
    bound, 6e-2 of the largest value, on the stream that the combine adds to), and captured and replayed."""
    H, I, E, k = 256, 256, 8, 2
    print(f"8-bit block serving step T={T}", flush=True)
    p = Layer(11, H, I, E)
    c1, s1 = moe.mxfp8_quantize(p.w1)
    c2, s2 = moe.mxfp8_quantize(p.w2)
    q = (c1, s1, c2, s2)
    x, y_in = _inputs(400, T, H)[:2]
    a, b, idx, prob, m = _serve(moe, p, x, y_in, q, k)
    om = oracle.permute(host(idx), E)
    pp = host(prob).astype(np.float64).ravel()[om["src_token"] * k + om["src_slot"]]
    rows = oracle.mxfp8_dequantize(host(a["codes"]), host(a["scales"]))[om["src_token"]]
    y = oracle.grouped_mlp_forward_mxfp8(rows, host(p.w1), host(p.w2), om["offsets"], pp)
    y = y[0] if isinstance(y, tuple) else y
    ref = oracle.add_rows(y, host(a["sum"]), host(m["row_id_map"]).reshape(T, k))
    assert np.abs(host(b["sum"]) - ref).max() <= 6e-2 * np.abs(ref).max()
    buf = [x.clone(), y_in.clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _serve(moe, p, *buf, q, k)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = _serve(moe, p, *buf, q, k)
    for rep in range(3):
        new = _inputs(500 + rep, T, H)[:2]
        for dst, src in zip(buf, new):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        got = [static[1][n].clone() for n in ("sum", "y", "codes", "scales")]
        eager = _serve(moe, p, *new, q, k)[1]
        torch.cuda.synchronize()
        for t, n in zip(got, ("sum", "y", "codes", "scales")):
            assert torch.equal(t, eager[n]), f"replay {rep}: {n}"
