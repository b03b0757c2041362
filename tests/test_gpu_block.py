"""One MoE block with everything around the experts, as a model's layer runs it: pre norm ->
router -> balance loss -> permute -> experts -> combine + post norm (+ the next layer's pre
norm), its whole backward, and the serving form with MXFP4 experts.

Training is compared with the float64 oracle stage by stage (each stage on the device's own
inputs, so that a stage's bound is that stage's) and end to end; then captured into a graph
and replayed, run on a side stream, and two captured blocks replayed at the same time.

End to end (bf16, float32 sums): dx is the sum of the residual's gradient and of what came
through the experts and the router; each bf16 tensor on the way rounds by at most 2^-8 of its
value and the roundings of different elements are independent, so the relative error of a
gradient tensor's norm stays below the sum over the roundings on its path (at most 10 tensors)
of 2^-8: 4e-2."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import host

pytestmark = pytest.mark.gpu

EPS, A, B = 1e-5, 0.01, 0.001
U = 2.0 ** -24
HALF = 2.0 ** -8


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
        self.wn1, self.wn2, self.wn3 = (bf(H, scale=0.1, mean=1.0) for _ in range(3))
        self.wr = bf(E, H, scale=H ** -0.5)
        self.w1, self.w2 = bf(E, 2 * I, H, scale=H ** -0.5), bf(E, H, I, scale=I ** -0.5)


def _inputs(seed, T, H, seqs):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    dout = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    gate = (1 + 0.2 * torch.randn((seqs, H), generator=g, device="cuda")).to(torch.bfloat16)
    mask = torch.rand(T, generator=g, device="cuda") < 0.9
    return x, dout, gate, mask


def _forward(moe, p, x, gate, mask, k, L):
    T = x.shape[0]
    a, r1 = moe.moe_pre_norm(x, p.wn1, EPS, save_rstd=True)
    logits = moe.moe_router_logits(a, p.wr)
    idx, prob = moe.moe_route_topk(logits, k)
    loss, counts, tokens = moe.moe_balance_loss(logits, idx, A, B, seq_len=L, mask=mask)
    m = moe.moe_permute(a, idx, prob, p.E)
    y, z, h = moe.moe_grouped_mlp_fwd(m["x_perm"], p.w1, p.w2, m["offsets"], m["prob_perm"], save_for_bwd=True)
    o = moe.moe_post_norm(y, x, p.wn2, row_id_map=m["row_id_map"], k=k, gate=gate, gate_group=L, eps=EPS,
                          save_for_bwd=True, next_weight=p.wn3)
    return dict(a=a, r1=r1, logits=logits, idx=idx, prob=prob, loss=loss, counts=counts, tokens=tokens, m=m, y=y, z=z, h=h, o=o)


def _backward(moe, p, f, x, dout, gate, mask, k, L):
    T = x.shape[0]
    m, o = f["m"], f["o"]
    post = moe.moe_post_norm_bwd(dout, o["c"], o["rstd"], p.wn2, row_id_map=m["row_id_map"], k=k, gate=gate, gate_group=L)
    dxp, dw1, dw2, dprob = moe.moe_grouped_mlp_bwd(post["dy"], m["x_perm"], f["z"], f["h"], m["prob_perm"], p.w1, p.w2,
                                                   m["offsets"])
    da = moe.moe_unpermute_combine(dxp, m["row_id_map"], T, k)
    dp = torch.index_select(dprob, 0, m["row_id_map"].long()).view(T, k)   # row order -> slots
    dl = moe.moe_route_topk_bwd(f["idx"], f["prob"], dp, p.E)
    dl = moe.moe_balance_loss_bwd(f["logits"], f["counts"], f["tokens"], k, A, B, seq_len=L, mask=mask, d_logits_in=dl,
                                  d_logits=dl)
    da, dwr = moe.moe_router_bwd(f["a"], p.wr, dl, dx_in=da)
    dx, dwn1 = moe.moe_pre_norm_bwd(da, x, p.wn1, f["r1"], dx_in=dout)
    return dict(dx=dx, dwn1=dwn1, dwn2=post["dweight"], dgate=post["dgate"], dwr=dwr, dw1=dw1, dw2=dw2, dl=dl, da=da,
                dy=post["dy"], dp=dp)


def _step(moe, p, inp, k, L):
    x, dout, gate, mask = inp
    f = _forward(moe, p, x, gate, mask, k, L)
    return f, _backward(moe, p, f, x, dout, gate, mask, k, L)


def _flat(f, b):
    return [f["o"]["out"], f["o"]["y_next"], f["loss"], f["counts"], *b.values()]


def _near(got, ref, mag, half, what):
    err = np.abs(host(got).astype(np.float64) - ref) / (half * np.abs(ref) + mag + 1e-30)
    assert np.all(err <= 1), f"{what}: {err.max():.2f} times the tolerance"


def _rel(got, ref):
    got = host(got).astype(np.float64)
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("T,H,I,E,k,L", [(96, 256, 256, 8, 2, 48), (65, 512, 256, 16, 4, 13), (1, 256, 256, 4, 1, 1)])
def test_training_step_against_the_oracle(moe, T, H, I, E, k, L):
    print(f"block training step T={T} H={H} I={I} E={E} k={k} L={L}", flush=True)
    p = Layer(T + H, H, I, E)
    inp = _inputs(T, T, H, T // L)
    x, dout, gate, mask = inp
    f, b = _step(moe, p, inp, k, L)
    X, D, G, M = host(x), host(dout), host(gate), host(mask)
    wn1, wn2, wn3, wr, w1, w2 = (host(t) for t in (p.wn1, p.wn2, p.wn3, p.wr, p.w1, p.w2))
    # stage by stage: the operators of this file's title on the device's own inputs
    a, r1 = oracle.pre_norm(X, wn1, EPS)
    _near(f["a"], a, 80 * U * np.abs(a), HALF, "pre norm")
    logits, idx = host(f["logits"]), host(f["idx"])
    loss, counts, tokens = oracle.balance_loss(logits, idx, A, B, L, M)[:3]
    assert np.array_equal(host(f["counts"]), counts)
    assert np.all(np.abs(host(f["loss"]) - loss) <= 256 * U * np.abs(loss) + 1e-12)
    rows = host(f["m"]["row_id_map"]).reshape(T, k)
    out, c, r2 = oracle.post_norm(host(f["y"]), X, wn2, EPS, rows, G, L)
    absc = oracle.post_norm(np.abs(host(f["y"])), X, wn2, EPS, rows)[1]
    g_all = np.abs(oracle.gate_rows(G, L, T, H))
    _near(f["o"]["out"], out, 80 * U * (np.abs(X) + g_all * r2[:, None] * np.abs(wn2) * absc), HALF, "out")
    u = oracle.pre_norm(host(f["o"]["out"]), wn3, EPS)[0]
    _near(f["o"]["y_next"], u, 80 * U * np.abs(u), HALF, "next norm")
    # end to end: the same chain in float64 from x, with the device's choice of experts
    lg = a @ wr.T
    e = np.exp(np.take_along_axis(lg, idx, 1) - np.take_along_axis(lg, idx, 1).max(1, keepdims=True))
    prob = e / e.sum(1, keepdims=True)
    m = oracle.permute(idx, E)
    src, slot = m["src_token"], m["src_slot"]
    rmap = np.asarray(m["row_id_map"]).reshape(T, k)
    assert np.array_equal(rmap, rows)
    xp, pp = a[src], prob.ravel()[src * k + slot]
    y = oracle.grouped_mlp_forward(xp, w1, w2, m["offsets"], pp)[0]
    out, c, r2 = oracle.post_norm(y, X, wn2, EPS, rows, G, L)
    assert _rel(f["o"]["out"], out) < 4e-2
    dc, dwn2, dgate = oracle.post_norm_backward(D, c, wn2, r2, G, L)
    dyp = dc[src]
    gb = oracle.grouped_mlp_backward(dyp, xp, w1, w2, m["offsets"], pp)
    dw1, dw2 = gb["dw_gate_up"], gb["dw_down"]
    da = np.zeros((T, H))
    np.add.at(da, src, gb["dx_perm"])
    dp = gb["dprob_perm"][rows]
    dl = oracle.route_topk_backward(lg, idx, dp) + oracle.balance_loss_backward(lg, idx, A, B, L, M)
    da_router, dwr = oracle.router_backward(a, wr, dl)
    da = da + da_router
    dx, dwn1 = oracle.pre_norm_backward(da, X, wn1, r1, D)
    for n, ref in (("dx", dx), ("dwn1", dwn1), ("dwn2", dwn2), ("dgate", dgate), ("dw1", dw1), ("dw2", dw2)):
        assert _rel(b[n], ref) < 4e-2, n
    if k > 1:   # with one expert a token the probabilities are 1 and only the balance loss reaches the router
        assert _rel(b["dwr"], dwr) < 4e-2


@pytest.mark.parametrize("seqs", [1, 4])
def test_training_step_graph_replays(moe, seqs):
    """Captured once, replayed on new inputs between eager runs, bit for bit the eager step."""
    T, H, I, E, k = 512, 512, 256, 16, 2
    L = T // seqs
    print(f"block training step under graph capture, {seqs} sequences", flush=True)
    p = Layer(3, H, I, E)
    buf = _inputs(100, T, H, seqs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(moe, p, buf, k, L)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = _flat(*_step(moe, p, buf, k, L))
    for rep in range(4):
        new = _inputs(200 + rep, T, H, seqs)
        for dst, src in zip(buf, new):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in static]
        ref = _flat(*_step(moe, p, new, k, L))
        torch.cuda.synchronize()
        for i, (s, r) in enumerate(zip(got, ref)):
            assert torch.equal(s.contiguous().view(torch.uint8), r.contiguous().view(torch.uint8)), f"replay {rep}: tensor {i}"


def test_two_streams_at_once(moe):
    """Two blocks in flight on two streams, each with its own workspaces, equal the same calls alone."""
    T, H, I, E, k, L = 1024, 512, 256, 16, 2, 256
    print("two blocks on two streams", flush=True)
    p = Layer(5, H, I, E)
    ins = [_inputs(300 + i, T, H, T // L) for i in range(2)]
    ref = [_flat(*_step(moe, p, i, k, L)) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for rep in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = _flat(*_step(moe, p, ins[i], k, L))
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(got[i], ref[i]):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def _serve(moe, p, x, q, k):
    """One serving layer: the norm before it was made by the layer before (post norm's next_weight)."""
    T = x.shape[0]
    a = moe.moe_pre_norm(x, p.wn1, EPS)
    idx, prob = moe.moe_route_topk(moe.moe_router_logits(a, p.wr), k)
    m = moe.moe_permute(a, idx, prob, p.E)
    y = moe.moe_grouped_mlp_fwd(m["x_perm"], q[0], q[2], m["offsets"], m["prob_perm"], compute="mxfp4", w_gate_up_scale=q[1],
                                w_down_scale=q[3])
    o = moe.moe_post_norm(y, x, p.wn2, row_id_map=m["row_id_map"], k=k, eps=EPS, next_weight=p.wn3)
    return o["out"], o["y_next"], idx, prob, m["row_id_map"], m["offsets"], a


@pytest.mark.parametrize("T", [1, 7, 64, 700])
def test_serving_step(moe, T):
    """MXFP4 experts: against the oracle with the same codes, and captured and replayed.

    The oracle quantises the float64 value of h where the kernel quantises its float32 value: a
    code may move to the neighbouring one (half a step of E2M1 at most 2^-2 relative, for the few
    values that lie that close to a boundary), so the output's norm is compared: 2e-2."""
    H, I, E, k = 256, 256, 8, 2
    print(f"block serving step T={T}", flush=True)
    p = Layer(11, H, I, E)
    c1, s1 = moe.mxfp4_quantize(p.w1.view(E * 2 * I, H))
    c2, s2 = moe.mxfp4_quantize(p.w2.view(E * H, I))
    q = (c1.view(E, 2 * I, H // 2), s1.view(E, 2 * I, H // 32), c2.view(E, H, I // 2), s2.view(E, H, I // 32))
    x = _inputs(400, T, H, 1)[0]
    out, u, idx, prob, rmap, off, a = _serve(moe, p, x, q, k)
    m = oracle.permute(host(idx), E)
    pp = host(prob).astype(np.float64).ravel()[m["src_token"] * k + m["src_slot"]]
    v1, v2 = (oracle.mxfp4_dequantize(c.cpu().numpy(), s.cpu().numpy()) for c, s in ((q[0], q[1]), (q[2], q[3])))
    y = oracle.mxfp4_mlp_forward(host(a)[m["src_token"]], v1, v2, m["offsets"], pp)[0]
    ref = oracle.post_norm(y, host(x), host(p.wn2), EPS, host(rmap).reshape(T, k))[0]
    assert _rel(out, ref) < 2e-2
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = _serve(moe, p, x, q, k)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(again[0], out) and torch.equal(again[1], u)
    buf = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = _serve(moe, p, buf, q, k)
    for rep in range(3):
        new = _inputs(500 + rep, T, H, 1)[0]
        buf.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in static[:2]]
        ref = _serve(moe, p, new, q, k)
        torch.cuda.synchronize()
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]), f"replay {rep}"


def test_two_graphs_share_a_workspace(moe):
    """Two captured products replayed one after the other on one stream, with one workspace between
    them: each call leaves nothing in it that the other needs."""
    E, K, N = 8, 768, 512
    print("two graphs, one workspace", flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn((E * N, K), generator=g, device="cuda").to(torch.bfloat16)
    c, s = moe.mxfp4_quantize(w)
    c, s = c.view(E, N, K // 2), s.view(E, N, K // 32)
    Rs = (24, 900)
    xs = [torch.randn((R, K), generator=g, device="cuda").to(torch.bfloat16) for R in Rs]
    offs = [torch.linspace(0, R, E + 1, device="cuda").int() for R in Rs]
    ref = [moe.moe_grouped_linear_mxfp4(x, c, s, o) for x, o in zip(xs, offs)]
    from grouped_expert_gemm_amd import _lib
    need = max(moe.workspace_size(_lib.MOE_OP_LINEAR_MXFP4, _lib.MlpDesc(E, K, N, _lib.MOE_MXFP4, _lib.MOE_BF16, _lib.MOE_MXFP4, 0), R)
               for R in Rs)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x, o in zip(xs, offs):
        out = torch.empty((x.shape[0], N), dtype=torch.bfloat16, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_grouped_linear_mxfp4(x, c, s, o, out=out, workspace=ws)
        graphs.append(graph)
        outs.append(out)
    for rep in range(3):
        for i in (0, 1, 1, 0):
            outs[i].zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[i], ref[i]), f"replay {rep} of graph {i}"
            ws.fill_(0xA5)
