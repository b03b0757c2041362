"""Cases for timing the operators around the MoE expert block: the load-balance loss, the
norms before and after the block, and the MXFP4 quantisation and grouped MLP.

`own` chooses what `run` calls: the plain torch form of each operator, or the framework's.
"""
import math

import torch

own = False

FP4 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # E2M1 magnitudes by code


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one micro-batch of the tiny layer: a call whose launches are its cost
        dict(name="balance tiny", kind="balance", T=256, E=8, k=2, seqs=1, masked=False, d_in=False, z=False),
        # a Qwen3-sized router in training: four padded sequences, z-loss, the routing gradient joined in
        dict(name="balance padded batch", kind="balance", T=16384, E=128, k=8, seqs=4, masked=True, d_in=True, z=True),
        # the largest router the library takes, a long accumulated batch
        dict(name="balance large", kind="balance", T=131072, E=256, k=8, seqs=1, masked=False, d_in=True, z=True),
        # one generated token of a Qwen3-sized layer: combine, norm, residual and the next block's norm
        dict(name="norm one token", kind="norm", T=1, H=2048, k=8, dtype="bf16", gate="none", group=1, scale=1.0,
             next=True, train=False),
        # a training step's two norms at the Mixtral width, gate per channel, residual scaled
        dict(name="norm training", kind="norm", T=4096, H=4096, k=2, dtype="bf16", gate="channel", group=4096,
             scale=0.8, next=False, train=True),
        # a prompt of a Qwen3-sized layer, eight rows combined per token, the next norm in the same pass
        dict(name="norm prompt", kind="norm", T=16384, H=2048, k=8, dtype="bf16", gate="token", group=1, scale=1.0,
             next=True, train=False),
        # a float32 block of odd width without routing, gate per sequence and channel
        dict(name="norm float32 odd width", kind="norm", T=1999, H=1001, k=1, dtype="f32", gate="channel", group=250,
             scale=1.0, next=False, train=True),
        # a Mixtral expert's gate_up weight made ready for serving, and read back
        dict(name="mxfp4 weights", kind="quant", rows=28672, cols=4096),
        # one generated token of a Qwen3-sized layer
        dict(name="mxfp4 one token", kind="mlp", T=1, H=2048, I=768, E=128, k=8),
        # a batch of generated tokens through the down product of a Mixtral-sized layer
        dict(name="mxfp4 linear batch", kind="linear", T=48, K=14336, N=4096, E=8, k=2),
        # a prompt of a Qwen3-sized layer: many small experts of uneven load
        dict(name="mxfp4 prompt small experts", kind="mlp", T=16384, H=2048, I=768, E=128, k=8),
        # a prompt of a Mixtral-sized layer
        dict(name="mxfp4 prompt large experts", kind="mlp", T=8192, H=4096, I=14336, E=8, k=2),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(("balance", "norm", "norm", "quant", "linear", "mlp", "mlp"))
    if kind == "balance":
        E = _spread(rng, 2, 256)
        seqs = rng.choice((1, 1, 3, 8))
        T = _spread(rng, 1, 131072 // seqs) * seqs
        return dict(kind=kind, T=T, E=E, k=rng.randint(1, min(E, 8)), seqs=seqs, masked=rng.random() < 0.5,
                    d_in=rng.random() < 0.5, z=rng.random() < 0.5)
    if kind == "norm":
        k = rng.choice((1, 2, 4, 8))
        H = _spread(rng, 16, 1024) * 8 if rng.random() < 0.7 else _spread(rng, 64, 8192)
        T = _spread(rng, 1, max(1, min(16384, (1 << 26) // (H * (k + 1)))))
        return dict(kind=kind, T=T, H=H, k=k, dtype=rng.choice(("bf16", "bf16", "f32")),
                    gate=rng.choice(("none", "token", "channel")), group=rng.randint(1, T),
                    scale=rng.choice((1.0, 0.5)), next=rng.random() < 0.5, train=rng.random() < 0.5)
    if kind == "quant":
        cols = 32 * _spread(rng, 1, 448)
        return dict(kind=kind, rows=_spread(rng, 1, (1 << 27) // cols), cols=cols)
    E = _spread(rng, 1, 128)
    k = rng.randint(1, min(E, 8))
    if kind == "linear":
        K, N = 256 * _spread(rng, 1, 32), 256 * _spread(rng, 1, 32)
        E = min(E, max(k, (1 << 30) // (K * N)))
        return dict(kind=kind, T=_spread(rng, 1, 8192 // k), K=K, N=N, E=E, k=k)
    H, I = 256 * _spread(rng, 1, 16), 256 * _spread(rng, 1, 24)
    E = min(E, max(k, (1 << 29) // (3 * H * I)))
    return dict(kind=kind, T=_spread(rng, 1, 16384 // k), H=H, I=I, E=E, k=k)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _fp4_codes(x):
    """float32 [..., cols] -> (E2M1 codes 0..15 [..., cols], E8M0 bytes [..., cols/32]): one scale
    2^s per 32 values, s the smallest with max|block| <= 6 * 2^s; codes to nearest, ties to even."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1)
    m, e = torch.frexp(amax)                       # amax = m 2^e, m in [0.5, 1); 6 = 0.75 * 2^3
    s = torch.where(m <= 0.75, e - 3, e - 2).clamp(-127, 127)
    s = torch.where(amax == 0, torch.full_like(s, -127), s)
    a = torch.ldexp(b, -s[..., None]).abs()
    # the number of midpoints below a; a midpoint itself goes to the even code beside it
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8)
         + (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8)
         + (a > 5.0).to(torch.uint8))
    c = c + (torch.signbit(b).to(torch.uint8) << 3)
    return c.reshape(x.shape), (s + 127).to(torch.uint8)


def _fp4_pack(c):
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _fp4_values(codes, scales):
    """packed codes [..., cols/2] and scale bytes -> float32 [..., cols]"""
    lut = torch.tensor(FP4 + tuple(-v for v in FP4), device=codes.device)
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1)
    v = v.reshape(*scales.shape, 32)
    return torch.ldexp(v, scales.int()[..., None] - 127).reshape(*codes.shape[:-1], -1)


def _round4(x):
    c, s = _fp4_codes(x)
    return _fp4_values(_fp4_pack(c), s)


def _weights(g, E, N, K):
    """E bf16 weights N(0, 0.02^2) [N, K] as MXFP4 (laid out once, before serving)"""
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((E, N, K // 32), dtype=torch.uint8, device="cuda")
    per = max(1, (1 << 28) // (N * K))
    for e in range(0, E, per):
        n = min(per, E - e)
        w = (0.02 * torch.randn((n, N, K), generator=g, device="cuda")).bfloat16().float()
        c, s = _fp4_codes(w)
        codes[e:e + n], scales[e:e + n] = _fp4_pack(c), s
    return codes, scales


def _routing(g, T, E, k):
    """The plan of a batch: offsets on the GPU, and on the host the experts that got rows"""
    load = 0.35 * torch.randn((1, E), generator=g, device="cuda")  # uneven experts
    logits = torch.randn((T, E), generator=g, device="cuda") + load
    top = torch.topk(logits, k, dim=1)
    counts = torch.bincount(top.indices.reshape(-1), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    host = counts.tolist()
    prob = torch.softmax(top.values, 1).reshape(-1)
    prob = prob[torch.argsort(top.indices.reshape(-1), stable=True)].contiguous()
    at = torch.repeat_interleave(torch.arange(E, device="cuda"), counts)
    active = torch.nonzero(counts)[:, 0]
    seat = torch.cumsum((counts > 0).long(), 0) - 1
    plan = dict(active=active, slot=seat[at], pos=torch.arange(T * k, device="cuda") - offsets[at].long(),
                most=max(host), counts=host)
    return offsets, prob, plan


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    s = dict(case=case)
    if case["kind"] == "balance":
        T, E = case["T"], case["E"]
        s["logits"] = rand(T, E) + 0.5 * rand(1, E)
        s["idx"] = torch.topk(s["logits"], case["k"], dim=1).indices.int().contiguous()
        s["mask"] = None
        if case["masked"]:  # sequences padded at their ends
            L = T // case["seqs"]
            n = torch.randint(max(1, L // 2), L + 1, (case["seqs"], 1), generator=g, device="cuda")
            s["mask"] = (torch.arange(L, device="cuda")[None] < n).reshape(-1).to(torch.uint8).contiguous()
        s["d_in"] = 1e-6 * rand(T, E) if case["d_in"] else None
        s["d_loss"] = torch.rand(1, generator=g, device="cuda") + 0.5
    elif case["kind"] == "norm":
        T, H, k = case["T"], case["H"], case["k"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["x"], s["y"] = rand(T, H).to(dt), (0.3 * rand(T * k, H)).to(dt)
        s["w"], s["w2"] = (1 + 0.1 * rand(H)).to(dt), (1 + 0.1 * rand(H)).to(dt)
        s["rows"] = torch.randperm(T * k, generator=g, device="cuda").int() if k > 1 else None
        s["gate"] = None
        if case["gate"] == "token":
            s["gate"] = torch.sigmoid(rand(T)).to(dt)
        elif case["gate"] == "channel":
            s["gate"] = (0.5 + 0.1 * rand(-(-T // case["group"]), H)).to(dt)
        if case["train"]:
            s["du"], s["dout"] = rand(T, H).to(dt), rand(T, H).to(dt)
    elif case["kind"] == "quant":
        s["w"] = (0.02 * rand(case["rows"], case["cols"])).bfloat16()
    else:
        T, E, k = case["T"], case["E"], case["k"]
        s["offsets"], s["prob"], s["plan"] = _routing(g, T, E, k)
        if case["kind"] == "linear":
            s["x"] = rand(T * k, case["K"]).bfloat16()
            s["w1"], s["s1"] = _weights(g, E, case["N"], case["K"])
        else:
            s["x"] = rand(T * k, case["H"]).bfloat16()
            s["w1"], s["s1"] = _weights(g, E, 2 * case["I"], case["H"])
            s["w2"], s["s2"] = _weights(g, E, case["H"], case["I"])
    return s


EPS, BALANCE, ZLOSS = 1e-6, 0.01, 0.001


def run(s):
    c = s["case"]
    if own:
        return _own(s, c)
    return {"balance": _plain_balance, "norm": _plain_norm, "quant": _plain_quant, "linear": _plain_linear,
            "mlp": _plain_mlp}[c["kind"]](s, c)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own(s, c):
    import grouped_expert_gemm_amd as moe
    if c["kind"] == "balance":
        z, L = ZLOSS if c["z"] else 0.0, c["T"] // c["seqs"]
        loss, counts, tokens = moe.moe_balance_loss(s["logits"], s["idx"], BALANCE, z, seq_len=L, mask=s["mask"])
        d = moe.moe_balance_loss_bwd(s["logits"], counts, tokens, c["k"], BALANCE, z, seq_len=L, mask=s["mask"],
                                     d_loss=s["d_loss"], d_logits_in=s["d_in"])
        return dict(loss=loss, counts=counts, d_logits=d)
    if c["kind"] == "norm":
        group = c["group"] if c["gate"] == "channel" else None
        r = moe.moe_post_norm(s["y"], s["x"], s["w"], row_id_map=s["rows"], k=c["k"], gate=s["gate"],
                              gate_group=group, residual_scale=c["scale"], eps=EPS, save_for_bwd=c["train"],
                              next_weight=s["w2"] if c["next"] else None)
        out = dict(out=r["out"])
        if c["next"]:
            out["u"] = r["y_next"]
        if c["train"]:
            u, rstd = moe.moe_pre_norm(s["x"], s["w2"], EPS, save_rstd=True)
            b = moe.moe_post_norm_bwd(s["dout"], r["c"], r["rstd"], s["w"], row_id_map=s["rows"], k=c["k"],
                                      gate=s["gate"], gate_group=group)
            dx, dw2 = moe.moe_pre_norm_bwd(s["du"], s["x"], s["w2"], rstd, dx_in=s["dout"], dx_in_scale=c["scale"])
            out.update(pre=u, dy=b["dy"], dw=b["dweight"], dx=dx, dw2=dw2)
            if s["gate"] is not None:
                out["dgate"] = b["dgate"]
        return out
    if c["kind"] == "quant":
        return moe.mxfp4_dequantize(*moe.mxfp4_quantize(s["w"]))
    if c["kind"] == "linear":
        return moe.moe_grouped_linear_mxfp4(s["x"], s["w1"], s["s1"], s["offsets"])
    return moe.moe_grouped_mlp_fwd(s["x"], s["w1"], s["w2"], s["offsets"], s["prob"], compute="mxfp4",
                                   w_gate_up_scale=s["s1"], w_down_scale=s["s2"])


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _plain_balance(s, c):
    S, E, k = c["seqs"], c["E"], c["k"]
    l = s["logits"].reshape(S, -1, E)
    m = torch.ones(l.shape[:2], device=l.device) if s["mask"] is None else s["mask"].reshape(S, -1).float()
    top = l.amax(-1, keepdim=True)
    ex = torch.exp(l - top)
    den = ex.sum(-1, keepdim=True)
    p = ex / den
    lse = (top + torch.log(den))[..., 0]
    hot = torch.zeros((S, E), device=l.device, dtype=torch.int32)
    hot.scatter_add_(1, s["idx"].reshape(S, -1).long(), m.int().repeat_interleave(k, 1))
    n = m.sum(1)
    seqs = (n > 0).sum().clamp(min=1)
    n1 = n.clamp(min=1)[:, None]
    over = (hot.double() * E / (n1 * k).double() - 1).float()  # E f - 1, near zero for even loads
    mean_p = (p * m[..., None]).sum(1) / n1
    live = (n > 0).float()
    balance = ((over * mean_p).sum(-1) + mean_p.sum(-1)) @ live / seqs
    z = ((lse * lse * m).sum(1) / n1[:, 0]) @ live / seqs
    zc = ZLOSS if c["z"] else 0.0
    loss = torch.stack((BALANCE * balance + zc * z, balance, z))
    share = (p * over[:, None]).sum(-1, keepdim=True)
    d = p * (BALANCE * (over[:, None] - share) + 2 * zc * lse[..., None])
    d = (d * (m[..., None] * (s["d_loss"] / seqs) / n1[..., None])).reshape(-1, E)
    return dict(loss=loss, counts=hot, d_logits=d if s["d_in"] is None else d + s["d_in"])


def _plain_gate(s, c, T, H):
    if s["gate"] is None:
        return torch.ones((1, 1), device=s["x"].device)
    if c["gate"] == "token":
        return s["gate"].float()[:, None]
    return s["gate"].float().repeat_interleave(c["group"], 0)[:T]


def _plain_norm(s, c):
    T, H, k, dt = c["T"], c["H"], c["k"], s["x"].dtype
    x, w, gate = s["x"].float(), s["w"].float(), _plain_gate(s, c, T, H)
    y = s["y"].float()
    comb = (y if s["rows"] is None else y[s["rows"].long()]).reshape(T, k, H).sum(1)
    r = torch.rsqrt(comb.square().mean(-1, keepdim=True) + EPS)
    res = dict(out=(c["scale"] * x + gate * (comb * r * w)).to(dt))
    w2 = s["w2"].float()
    if c["next"]:
        o = res["out"].float()
        res["u"] = (o * torch.rsqrt(o.square().mean(-1, keepdim=True) + EPS) * w2).to(dt)
    if c["train"]:
        rx = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        xh = x * rx
        res["pre"] = (xh * w2).to(dt)
        ch = comb.to(dt).float() * r  # the stored sum
        dout = s["dout"].float()
        a = dout * ch
        if c["gate"] == "token":
            res["dgate"] = (a * w).sum(-1)
        elif c["gate"] == "channel":
            of = torch.arange(T, device=x.device) // c["group"]
            res["dgate"] = torch.zeros(s["gate"].shape, device=x.device).index_add_(0, of, a * w)
        res["dw"] = (a * gate).sum(0)
        dn = dout * gate * w
        dc = (r * (dn - ch * (dn * ch).mean(-1, keepdim=True))).to(dt)
        if s["rows"] is None:
            res["dy"] = dc
        else:
            res["dy"] = torch.empty((T * k, H), dtype=dt, device=x.device)
            res["dy"][s["rows"].long()] = dc.repeat_interleave(k, 0)
        du = s["du"].float()
        res["dw2"] = (du * xh).sum(0)
        dn = du * w2
        res["dx"] = (c["scale"] * dout + rx * (dn - xh * (dn * xh).mean(-1, keepdim=True))).to(dt)
    return res


def _plain_quant(s, c):
    return _round4(s["w"].float()).bfloat16()


def _plain_product(x, codes, scales, plan):
    """x [R, K] float32 times each row's expert [N, K], the rows of the experts that have some side by side"""
    w = _fp4_values(codes[plan["active"]], scales[plan["active"]])
    padded = torch.zeros((w.shape[0], plan["most"], x.shape[1]), device=x.device)
    padded[plan["slot"], plan["pos"]] = x
    y = torch.bmm(w, padded.transpose(1, 2).contiguous())
    return y.transpose(1, 2)[plan["slot"], plan["pos"]]


def _plain_linear(s, c):
    return _plain_product(_round4(s["x"].float()), s["w1"], s["s1"], s["plan"]).bfloat16()


def _plain_mlp(s, c):
    z = _plain_product(_round4(s["x"].float()), s["w1"], s["s1"], s["plan"])
    gate, up = z[:, :c["I"]], z[:, c["I"]:]
    h = gate / (1 + torch.exp(-gate)) * up * s["prob"][:, None]
    return _plain_product(_round4(h), s["w2"], s["s2"], s["plan"]).bfloat16()


# ---------------------------------------------------------------------------
# what one pass reads, writes and computes
# ---------------------------------------------------------------------------

def work(case):
    c = case
    if c["kind"] == "balance":
        T, E, k = c["T"], c["E"], c["k"]
        once = 4 * T * E + 4 * T * k + (T if c["masked"] else 0)
        return dict(bytes=once + 4 * T * E * (3 if c["d_in"] else 2), flops=20 * T * E)
    if c["kind"] == "norm":
        T, H, k = c["T"], c["H"], c["k"]
        e = 2 if c["dtype"] == "bf16" else 4
        rows = T * k + 2 * T + (T if c["next"] else 0)
        if c["train"]:
            rows += T + 2 * T          # the stored sum, the pre norm
            rows += 2 * T + T * k      # post norm backward
            rows += 4 * T              # pre norm backward
        return dict(bytes=rows * H * e, flops=10 * rows * H)
    if c["kind"] == "quant":
        n = c["rows"] * c["cols"]
        return dict(bytes=2 * n + 2 * (n // 2 + n // 32) + 2 * n, flops=10 * n)
    R, E = c["T"] * c["k"], c["E"]
    used = E * (1 - (1 - c["k"] / E) ** c["T"])  # experts that get rows, for even loads
    per = 0.5 + 1 / 32
    if c["kind"] == "linear":
        return dict(bytes=used * c["K"] * c["N"] * per + 2 * R * (c["K"] + c["N"]), flops=2 * R * c["K"] * c["N"])
    n = 3 * c["H"] * c["I"]
    return dict(bytes=used * n * per + 4 * R * c["H"], flops=2 * R * n)


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _exact_round4(x):
    """Each value of [..., cols] as the nearest of the 15 E2M1 values times its block's scale"""
    b = x.double().reshape(-1, 32)
    top = b.abs().max(1, keepdim=True).values
    s = torch.ceil(torch.log2((top / 6).clamp(min=2.0 ** -140)))
    s = torch.where(top > 6 * torch.exp2(s), s + 1, torch.where(top <= 6 * torch.exp2(s - 1), s - 1, s))
    s = s.clamp(-127, 127)
    grid = torch.tensor(FP4, dtype=torch.float64, device=x.device)
    a = b.abs() / torch.exp2(s)
    hi = torch.searchsorted(grid, a.contiguous()).clamp(1, 7)
    lo = hi - 1
    up, down = grid[hi] - a, a - grid[lo]
    pick = torch.where(up < down, hi, torch.where(down < up, lo, torch.where(hi % 2 == 0, hi, lo)))
    return torch.copysign(grid[pick] * torch.exp2(s), b).reshape(x.shape)


def _exact_weight(codes, scales):
    grid = torch.tensor(FP4, dtype=torch.float64, device=codes.device)
    n, half = codes.shape
    v = torch.empty((n, 2 * half), dtype=torch.float64, device=codes.device)
    v[:, 0::2] = grid[(codes % 8).long()] * (1 - 2.0 * (codes // 8 % 2))
    v[:, 1::2] = grid[(codes // 16 % 8).long()] * (1 - 2.0 * (codes // 128))
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    f = lambda t: t.double()  # noqa: E731
    if c["kind"] == "balance":
        S, E, L = c["seqs"], c["E"], c["T"] // c["seqs"]
        zc = ZLOSS if c["z"] else 0.0
        d = torch.zeros((c["T"], E), dtype=torch.float64, device="cuda")
        total = torch.zeros(3, dtype=torch.float64, device="cuda")
        counts, parts = [], []
        for q in range(S):
            keep = torch.ones(L, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"][q * L:(q + 1) * L] > 0
            at = torch.nonzero(keep)[:, 0] + q * L
            cnt = torch.bincount(s["idx"][at].reshape(-1).long(), minlength=E)
            counts.append(cnt)
            if at.numel():
                parts.append((at, cnt))
        for at, cnt in parts:
            l = f(s["logits"][at])
            p, lse = torch.softmax(l, 1), torch.logsumexp(l, 1)
            frac = f(cnt) / (c["k"] * at.numel())
            b, z = E * (frac * p.mean(0)).sum(), (lse ** 2).mean()
            total += torch.stack((BALANCE * b + zc * z, b, z)) / len(parts)
            inner = BALANCE * E * (frac - (p * frac).sum(1, keepdim=True)) + 2 * zc * lse[:, None]
            d[at] = p * inner * f(s["d_loss"]) / (len(parts) * at.numel())
        if s["d_in"] is not None:
            d += f(s["d_in"])
        return dict(loss=total, counts=torch.stack(counts).int(), d_logits=d)
    if c["kind"] == "norm":
        T, H, k = c["T"], c["H"], c["k"]
        x, w, w2 = f(s["x"]), f(s["w"]), f(s["w2"])
        comb = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        for j in range(k):
            comb += f(s["y"]) if s["rows"] is None else f(s["y"])[s["rows"].reshape(T, k)[:, j].long()]
        r = 1 / torch.sqrt((comb * comb).sum(1, keepdim=True) / H + EPS)
        if c["gate"] == "none":
            gate = torch.ones((T, H), dtype=torch.float64, device="cuda")
        elif c["gate"] == "token":
            gate = f(s["gate"])[:, None].expand(T, H)
        else:
            gate = f(s["gate"])[torch.arange(T, device="cuda") // c["group"]]
        out = c["scale"] * x + gate * w * comb * r
        res = dict(out=out)
        if c["next"]:
            o = f(out.to(s["x"].dtype))  # the next norm reads the stored sum
            res["u"] = o / torch.sqrt((o * o).sum(1, keepdim=True) / H + EPS) * w2
        if c["train"]:
            rx = 1 / torch.sqrt((x * x).sum(1, keepdim=True) / H + EPS)
            res["pre"] = x * rx * w2
            ch = f(comb.to(s["x"].dtype)) * r  # the backward reads the stored sum
            dout, du = f(s["dout"]), f(s["du"])
            res["dw"] = (dout * gate * ch).sum(0)
            if c["gate"] == "token":
                res["dgate"] = (dout * w * ch).sum(1)
            elif c["gate"] == "channel":
                res["dgate"] = torch.stack([(dout * w * ch)[t:t + c["group"]].sum(0) for t in range(0, T, c["group"])])
            a = dout * gate * w
            dc = r * a - r * ch * (a * ch).sum(1, keepdim=True) / H
            if s["rows"] is None:
                res["dy"] = dc
            else:
                res["dy"] = torch.zeros((T * k, H), dtype=torch.float64, device="cuda")
                for j in range(k):
                    res["dy"][s["rows"].reshape(T, k)[:, j].long()] = dc
            a, xh = du * w2, x * rx
            res["dw2"] = (du * xh).sum(0)
            res["dx"] = c["scale"] * dout + rx * a - rx * xh * (a * xh).sum(1, keepdim=True) / H
        return res
    if c["kind"] == "quant":
        return _exact_round4(s["w"])
    xq = _exact_round4(s["x"])
    y = torch.zeros((xq.shape[0], c["N"] if c["kind"] == "linear" else c["H"]), dtype=torch.float64, device="cuda")
    at = 0
    for e, n in enumerate(s["plan"]["counts"]):
        if not n:
            continue
        z = xq[at:at + n] @ _exact_weight(s["w1"][e], s["s1"][e]).T
        if c["kind"] == "linear":
            y[at:at + n] = z
        else:
            gate, up = z[:, :c["I"]], z[:, c["I"]:]
            h = gate * torch.sigmoid(gate) * up * f(s["prob"][at:at + n, None])
            y[at:at + n] = _exact_round4(h) @ _exact_weight(s["w2"][e], s["s2"][e]).T
        at += n
    return y
