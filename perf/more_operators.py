"""Cases for timing the operators that hold a block's activations in 8 bits: the norm that adds
the residual and writes MXFP8 rows, the reading of MXFP8 rows, and the grouped MLP whose
forward keeps its gate_up output in MXFP8 and whose backward works from what was kept.

`own` chooses what `run` calls: the plain torch form of each operator, or the framework's.
"""
import math

import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one generated token between two Qwen3-sized blocks: its eight expert rows combined, added to
        # the residual and normalised, for the router (y) and for MXFP8 experts
        dict(name="norm8 one token", kind="norm8", T=1, H=2048, k=8, dtype="bf16", residual=True, y=True),
        # a prompt through the same place
        dict(name="norm8 prompt", kind="norm8", T=16384, H=2048, k=8, dtype="bf16", residual=True, y=True),
        # a training step's norm at the Mixtral width: the attention's output added, codes kept for the backward
        dict(name="norm8 training", kind="norm8", T=8192, H=4096, k=1, dtype="bf16", residual=True, y=True),
        # a float32 residual stream of odd width, codes only
        dict(name="norm8 float32 odd width", kind="norm8", T=1999, H=1056, k=1, dtype="f32", residual=True, y=False),
        # a layer's kept rows read back in the order of its experts
        dict(name="read8 by token", kind="read8", rows=4096, cols=4096, k=2),
        # a few kept rows of odd width, in their own order
        dict(name="read8 odd", kind="read8", rows=77, cols=1440, k=0),
        # a training step of the small layer: a call whose launches are its cost
        dict(name="forward small", kind="fwd", T=256, H=256, I=256, E=8, k=2),
        # a Qwen3-sized layer: many small experts of uneven load
        dict(name="forward small experts", kind="fwd", T=16384, H=2048, I=768, E=128, k=8),
        # a Mixtral-sized layer
        dict(name="forward large experts", kind="fwd", T=4096, H=4096, I=14336, E=8, k=2),
        # the backward of the same three layers
        dict(name="backward small", kind="bwd", T=256, H=256, I=256, E=8, k=2),
        dict(name="backward small experts", kind="bwd", T=16384, H=2048, I=768, E=128, k=8),
        dict(name="backward large experts", kind="bwd", T=4096, H=4096, I=14336, E=8, k=2),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    kind = rng.choice(("norm8", "norm8", "read8", "fwd", "fwd", "bwd", "bwd"))
    if kind == "norm8":
        k = rng.choice((1, 1, 2, 8))
        H = 32 * _spread(rng, 1, 512)
        T = _spread(rng, 1, max(1, min(16384, (1 << 26) // (H * k))))
        return dict(kind=kind, T=T, H=H, k=k, dtype=rng.choice(("bf16", "bf16", "f32")),
                    residual=rng.random() < 0.8, y=rng.random() < 0.5)
    if kind == "read8":
        cols = 32 * _spread(rng, 1, 512)
        k = rng.choice((0, 1, 2, 8))
        return dict(kind=kind, rows=_spread(rng, 1, max(1, (1 << 26) // (cols * max(k, 1)))), cols=cols, k=k)
    E = _spread(rng, 1, 128)
    k = rng.randint(1, min(E, 8))
    H, I = 256 * _spread(rng, 1, 16), 256 * _spread(rng, 1, 24)
    E = min(E, max(k, (1 << 29) // (3 * H * I)))
    return dict(kind=kind, T=_spread(rng, 1, 16384 // k), H=H, I=I, E=E, k=k)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _mx8(x):
    """float32 [rows, cols] -> (E4M3 codes [rows, cols] uint8, E8M0 bytes [rows, cols/32] uint8): one scale
    2^s per 32 values, s the smallest with max|block| <= 448 * 2^s; codes to nearest, ties to even."""
    b = x.reshape(x.shape[0], -1, 32)
    amax = b.abs().amax(-1)
    m, e = torch.frexp(amax)                       # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    s = torch.where(m <= 0.875, e - 9, e - 8).clamp(-127, 127)
    s = torch.where(amax == 0, torch.full_like(s, -127), s)
    c = torch.ldexp(b, -s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return c.reshape(x.shape), (s + 127).to(torch.uint8)


def _mx8_values(codes, scales):
    """codes [rows, cols] and scale bytes [rows, cols/32] -> float32 [rows, cols]"""
    v = codes.view(torch.float8_e4m3fn).float().reshape(codes.shape[0], -1, 32)
    return torch.ldexp(v, scales.int()[..., None] - 127).reshape(codes.shape)


def _weights(g, E, N, K):
    w = torch.empty((E, N, K), dtype=torch.bfloat16, device="cuda")
    per = max(1, (1 << 28) // (N * K))
    for e in range(0, E, per):
        w[e:e + per] = 0.02 * torch.randn((min(per, E - e), N, K), generator=g, device="cuda")
    return w


def _routing(g, T, E, k):
    """The plan of a batch: offsets, routing weights and tokens of the grouped rows on the GPU, and the rows per expert"""
    load = 0.35 * torch.randn((1, E), generator=g, device="cuda")  # uneven experts
    top = torch.topk(torch.randn((T, E), generator=g, device="cuda") + load, k, dim=1)
    idx = top.indices.reshape(-1)
    order = torch.argsort(idx, stable=True)
    counts = torch.bincount(idx, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    prob = torch.softmax(top.values, 1).reshape(-1)[order].contiguous()
    at = torch.repeat_interleave(torch.arange(E, device="cuda"), counts)
    seat = torch.cumsum((counts > 0).long(), 0) - 1
    host = counts.tolist()
    plan = dict(active=torch.nonzero(counts)[:, 0], slot=seat[at], most=max(host), counts=host,
                pos=torch.arange(T * k, device="cuda") - offsets[at].long())
    return offsets, prob, (order // k).int(), plan


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    c, s = case, dict(case=case)
    if c["kind"] == "norm8":
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        s["x"] = (0.3 * rand(c["T"] * c["k"], c["H"])).to(dt)
        s["residual"] = rand(c["T"], c["H"]).to(dt) if c["residual"] else None
        s["w"] = (1 + 0.1 * rand(c["H"])).to(dt)
        s["rows"] = torch.randperm(c["T"] * c["k"], generator=g, device="cuda").int() if c["k"] > 1 else None
    elif c["kind"] == "read8":
        s["codes"], s["scales"] = _mx8(rand(c["rows"], c["cols"]) * torch.exp(2 * rand(c["rows"], 1)))
        s["rows"] = None
        if c["k"]:
            s["rows"] = torch.randperm(c["rows"] * c["k"], generator=g, device="cuda").int() // c["k"]
    else:
        T, H, I, E = c["T"], c["H"], c["I"], c["E"]
        s["offsets"], s["prob"], s["src"], s["plan"] = _routing(g, T, E, c["k"])
        s["w1"], s["w2"] = _weights(g, E, 2 * I, H), _weights(g, E, H, I)
        if c["kind"] == "fwd":
            s["x"] = rand(T, H).bfloat16()[s["src"].long()]
        else:  # what the forward kept, and the gradient that comes back
            s["xc"], s["xs"] = _mx8(rand(T, H))
            s["zc"], s["zs"] = _mx8(0.02 * math.sqrt(H) * rand(T * c["k"], 2 * I))
            s["dy"] = rand(T, H).bfloat16()[s["src"].long()]
    return s


def run(s):
    c = s["case"]
    if own:
        return _own(s, c)
    return {"norm8": _plain_norm8, "read8": _plain_read8, "fwd": _plain_fwd, "bwd": _plain_bwd}[c["kind"]](s, c)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own(s, c):
    import grouped_expert_gemm_amd as moe
    if c["kind"] == "norm8":
        r = moe.moe_add_norm_mxfp8(s["x"], s["w"], residual=s["residual"], row_id_map=s["rows"], k=c["k"], eps=EPS,
                                   with_y=c["y"], save_for_bwd=True)
        out = dict(sum=r["sum"], rstd=r["rstd"], values=moe.mxfp8_dequantize(r["codes"], r["scales"]))
        if c["y"]:
            out["y"] = r["y"]
        return out
    if c["kind"] == "read8":
        return moe.mxfp8_dequantize(s["codes"], s["scales"], src_row=s["rows"])
    if c["kind"] == "fwd":
        y, zc, zs = moe.moe_grouped_mlp_fwd_ckpt8(s["x"], s["w1"], s["w2"], s["offsets"], s["prob"])
        return dict(y=y, z=moe.mxfp8_dequantize(zc, zs))
    dx, dw1, dw2, dprob = moe.moe_grouped_mlp_bwd_ckpt8(s["dy"], s["xc"], s["zc"], s["zs"], s["prob"], s["w1"], s["w2"],
                                                        s["offsets"], x_scale=s["xs"], src_token=s["src"])
    return dict(dx=dx, dw1=dw1, dw2=dw2, dprob=dprob)


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _plain_norm8(s, c):
    x, dt = s["x"].float(), s["x"].dtype
    total = (x if s["rows"] is None else x[s["rows"].long()]).reshape(c["T"], c["k"], c["H"]).sum(1)
    if s["residual"] is not None:
        total = s["residual"].float() + total
    kept = total.to(dt)
    v = kept.float()
    rstd = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    n = v * rstd * s["w"].float()
    out = dict(sum=kept, rstd=rstd[:, 0], values=_mx8_values(*_mx8(n)).bfloat16())
    if c["y"]:
        out["y"] = n.to(dt)
    return out


def _plain_read8(s, c):
    v = _mx8_values(s["codes"], s["scales"]).bfloat16()
    return v if s["rows"] is None else v[s["rows"].long()]


def _padded(x, plan):
    """rows [R, n] side by side for each expert that has some: [experts, most rows, n], zeros behind"""
    p = torch.zeros((plan["active"].shape[0], plan["most"], x.shape[1]), device=x.device)
    p[plan["slot"], plan["pos"]] = x
    return p


def _flat(p, plan):
    return p[plan["slot"], plan["pos"]]


def _times(x, w, plan):
    """x [R, K] float32 times each row's expert, w [experts, K, N] contiguous"""
    return _flat(torch.bmm(_padded(x, plan), w), plan)


def _silu_parts(z, I):
    g, u = z[:, :I], z[:, I:]
    sig = 1 / (1 + torch.exp(-g))
    return g, u, sig


def _plain_fwd(s, c):
    plan = s["plan"]
    z = _times(s["x"].float(), s["w1"][plan["active"]].float().transpose(1, 2).contiguous(), plan)
    g, u, sig = _silu_parts(z, c["I"])
    h = g * sig * u * s["prob"][:, None]
    y = _times(h, s["w2"][plan["active"]].float().transpose(1, 2).contiguous(), plan)
    return dict(y=y.bfloat16(), z=_mx8_values(*_mx8(z)).bfloat16())


def _plain_weight_grad(a, b, plan, shape):
    """sum over each expert's rows of a[r]^T b[r], in bf16; zeros for experts without rows"""
    dw = torch.zeros(shape, dtype=torch.bfloat16, device=a.device)
    dw[plan["active"]] = torch.bmm(_padded(a, plan).transpose(1, 2).contiguous(), _padded(b, plan)).bfloat16()
    return dw


def _plain_bwd(s, c):
    plan, I, p = s["plan"], c["I"], s["prob"][:, None]
    x = _mx8_values(s["xc"], s["xs"])[s["src"].long()]
    g, u, sig = _silu_parts(_mx8_values(s["zc"], s["zs"]), I)
    dy = s["dy"].float()
    dh = _times(dy, s["w2"][plan["active"]].float(), plan)
    act = g * sig
    dprob = (dh * act * u).sum(1)
    dz = torch.cat((dh * p * u * sig * (1 + g * (1 - sig)), dh * p * act), 1)
    dx = _times(dz, s["w1"][plan["active"]].float(), plan)
    dw1 = _plain_weight_grad(dz, x, plan, s["w1"].shape)
    dw2 = _plain_weight_grad(dy, act * u * p, plan, s["w2"].shape)
    return dict(dx=dx.bfloat16(), dw1=dw1, dw2=dw2, dprob=dprob)


# ---------------------------------------------------------------------------
# what one pass reads, writes and computes
# ---------------------------------------------------------------------------

def work(case):
    c = case
    per = 1 + 1 / 32  # bytes of a value in MXFP8
    if c["kind"] == "norm8":
        T, H, k = c["T"], c["H"], c["k"]
        e = 2 if c["dtype"] == "bf16" else 4
        rows = k + int(c["residual"]) + 1 + int(c["y"])
        # the codes are written, and read back as the bf16 values that the pass returns
        return dict(bytes=T * H * (rows * e + 2 * per + 2), flops=(k + 12) * T * H)
    if c["kind"] == "read8":
        n, out = c["rows"] * c["cols"], c["rows"] * max(c["k"], 1) * c["cols"]
        return dict(bytes=n * per + 2 * out + (4 * out // c["cols"] if c["k"] else 0), flops=out)
    T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    R = T * k
    used = E * (1 - (1 - k / E) ** T)  # experts that get rows, for even loads
    weights = 6 * H * I
    if c["kind"] == "fwd":
        return dict(bytes=used * weights + 4 * R * H + 2 * R * I * (2 * per + 2), flops=6 * R * H * I)
    return dict(bytes=used * weights + E * weights + 4 * R * H + per * (T * H + 2 * R * I) + 12 * R, flops=12 * R * H * I)


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _exact_mx8(x):
    """Each value of float64 [rows, cols] as the nearest E4M3 value times its block's power of two"""
    b = x.reshape(-1, 32)
    top = b.abs().max(1, keepdim=True).values
    s = torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** -140)))
    s = torch.where(top > 448 * torch.exp2(s), s + 1, torch.where(top <= 448 * torch.exp2(s - 1), s - 1, s))
    s = s.clamp(-127, 127)
    a = b / torch.exp2(s)
    step = torch.exp2(torch.floor(torch.log2(a.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(a / step) * step * torch.exp2(s)).reshape(x.shape)


def _exact_values(codes, scales):
    c = codes.long()
    e, m = c // 8 % 16, (c % 8).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(e.double() - 7)) * (1 - 2.0 * (c // 128).double())
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    f = lambda t: t.double()  # noqa: E731
    if c["kind"] == "norm8":
        total = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device="cuda")
        for j in range(c["k"]):
            total += f(s["x"]) if s["rows"] is None else f(s["x"])[s["rows"].reshape(c["T"], -1)[:, j].long()]
        if s["residual"] is not None:
            total += f(s["residual"])
        v = f(total.to(s["x"].dtype))  # the norm reads the sum as it is stored
        r = 1 / torch.sqrt((v * v).sum(1, keepdim=True) / c["H"] + EPS)
        n = v * r * f(s["w"])
        out = dict(sum=total, rstd=r[:, 0], values=_exact_mx8(n))
        if c["y"]:
            out["y"] = n
        return out
    if c["kind"] == "read8":
        v = _exact_values(s["codes"], s["scales"])
        return v if s["rows"] is None else v.index_select(0, s["rows"].long())
    I, H, R = c["I"], c["H"], c["T"] * c["k"]
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    at, out = 0, None
    if c["kind"] == "fwd":
        out = dict(y=new(R, H), z=new(R, 2 * I))
    else:
        out = dict(dx=new(R, H), dw1=torch.zeros_like(s["w1"], dtype=torch.float64),
                   dw2=torch.zeros_like(s["w2"], dtype=torch.float64), dprob=new(R))
    for e, n in enumerate(s["plan"]["counts"]):
        if not n:
            continue
        to, p = slice(at, at + n), f(s["prob"][at:at + n, None])
        w1, w2 = f(s["w1"][e]), f(s["w2"][e])
        if c["kind"] == "fwd":
            z = f(s["x"][to]) @ w1.T
            out["y"][to] = (z[:, :I] * torch.sigmoid(z[:, :I]) * z[:, I:] * p) @ w2.T
            out["z"][to] = _exact_mx8(z)
        else:
            z = _exact_values(s["zc"][to], s["zs"][to])
            src = s["src"][to].long()
            x, dy = _exact_values(s["xc"][src], s["xs"][src]), f(s["dy"][to])
            g, u = z[:, :I], z[:, I:]
            sig = torch.sigmoid(g)
            dh = dy @ w2
            out["dprob"][to] = (dh * g * sig * u).sum(1)
            dz = torch.cat((dh * u * p * (sig + g * sig * (1 - sig)), dh * p * g * sig), 1)
            out["dx"][to] = dz @ w1
            out["dw1"][e] = dz.T @ x
            out["dw2"][e] = dy.T @ (g * sig * u * p)
        at += n
    return out
