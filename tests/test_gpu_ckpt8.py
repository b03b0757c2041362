"""GPU parity of the bf16 grouped MLP over 8-bit checkpoints, forward and backward, against the
float64 oracle.

Tolerances (u = 2^-24, float32's half step; h = 2^-8, bf16's), as bounds on sums of magnitudes:
- a float32 sum of n products is off by at most n u of the sum of their magnitudes, in any order;
- z is such a sum over H; its codes may be any that a value within that of the exact one
  rounds to (rounding is monotone: those between the codes of the interval's ends);
- silu and sigmoid take a hardware exponential and reciprocal (2 and 1 units) and a few products:
  16 u of the value, of sig + silu (1 - sig) by 16 u of the sum of its magnitudes;
- h and dZ are rounded once to bf16 (h of the value) before the products that read them, whose
  float32 sums and final rounding come on top."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from gpu_util import host

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = 2.0 ** -8


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import grouped_expert_gemm_amd as g
    g.lib()
    return g


class Case:
    """Random operands: counts rows for each expert and `behind` rows past the last one's."""

    def __init__(self, counts, H, I, seed, behind=0, k=2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.counts, self.H, self.I, self.E = counts, H, I, len(counts)
        self.used = sum(counts)
        self.R = self.used + behind
        self.T = max(1, -(-self.R // k))
        self.off_host = np.concatenate([[0], np.cumsum(counts)])
        self.offsets = torch.tensor(self.off_host, dtype=torch.int32, device="cuda")
        self.w1 = (H ** -0.5 * n(self.E, 2 * I, H)).bfloat16()
        self.w2 = (I ** -0.5 * n(self.E, H, I)).bfloat16()
        self.x = n(self.R, H).bfloat16()
        self.dy = n(self.R, H).bfloat16()
        self.prob = torch.rand(self.R, generator=g, device="cuda") + 0.1
        self.src = torch.randint(0, self.T, (self.R,), generator=g, device="cuda").int()
        self.tokens = n(self.T, H).bfloat16()


def _forward_check(moe, c):
    y, zc, zs = moe.moe_grouped_mlp_fwd_ckpt8(c.x, c.w1, c.w2, c.offsets, c.prob)
    codes, scales = host(zc)[:c.used], host(zs)[:c.used]
    x, w1 = host(c.x), host(c.w1)
    z, mag = np.zeros((c.used, 2 * c.I)), np.zeros((c.used, 2 * c.I))
    for e in range(c.E):
        r = slice(c.off_host[e], c.off_host[e + 1])
        z[r], mag[r] = x[r] @ w1[e].T, np.abs(x[r]) @ np.abs(w1[e]).T
    if c.used:
        lo, hi, ok = oracle.mxfp8_bounds(z, c.H * U * mag, scales)
        v = oracle.mxfp8_dequantize(codes, scales)
        assert ok.all(), "scale bytes of z"
        assert np.all((lo <= v) & (v <= hi)), "codes of z"
    got, w2, p = host(y), host(c.w2), host(c.prob).astype(np.float64)
    for e in range(c.E):
        r = slice(c.off_host[e], c.off_host[e + 1])
        g, u, pe = z[r, :c.I], z[r, c.I:], p[r, None]
        sig = 1 / (1 + np.exp(-np.clip(g, -700, None)))
        h, ez = g * sig * u * pe, c.H * U * mag[r]
        slope = sig + np.abs(g) * sig * (1 - sig)                       # of silu; h moves with z's error
        eh = (HALF + 20 * U) * np.abs(h) + (1 + HALF) * pe * (slope * np.abs(u) * ez[:, :c.I] + np.abs(g * sig) * ez[:, c.I:])
        ref, w = h @ w2[e].T, np.abs(w2[e]).T
        tol = HALF * np.abs(ref) + (1 + HALF) * (eh @ w + c.I * U * (np.abs(h) + eh) @ w) + 1e-30
        assert np.all(np.abs(got[r] - ref) <= tol), f"y of expert {e}"
        assert np.linalg.norm(got[r] - ref) <= 2 * HALF * np.linalg.norm(ref), f"y of expert {e} (norm)"
    return zc, zs


def _backward_check(moe, c, zc, zs, got, xv, what):
    """got: (dx, dw1, dw2, dprob); xv: the values of x in expert order (host)"""
    n = c.used
    z = np.zeros((c.R, 2 * c.I))
    if n:
        z[:n] = oracle.mxfp8_dequantize(host(zc)[:n], host(zs)[:n])
    w1, w2, dy, p = host(c.w1), host(c.w2), host(c.dy), host(c.prob).astype(np.float64)
    ref = oracle.grouped_mlp_backward_from_z(dy, xv, z, w1, w2, c.off_host, p)
    dx, dw1, dw2, dprob = (host(t).astype(np.float64) for t in got)
    I, H = c.I, c.H
    g, u = z[:, :I], z[:, I:]
    sig = 1 / (1 + np.exp(-np.clip(g, -700, None)))
    act, fg, fu = np.abs(g * sig), np.abs(p[:, None] * u) * (sig + np.abs(g) * sig * (1 - sig)), np.abs(p[:, None] * g * sig)
    for e in range(c.E):
        r = slice(c.off_host[e], c.off_host[e + 1])
        if r.start == r.stop:
            assert not dw1[e].any() and not dw2[e].any(), f"{what}: gradients of an idle expert"
            continue
        m = r.stop - r.start
        dh, dhm = dy[r] @ w2[e], np.abs(dy[r]) @ np.abs(w2[e])
        edh = H * U * dhm                                                  # dH's float32 sum
        tol = (np.abs(dh) * 16 * U + edh) * act[r] * np.abs(u[r])
        tol = tol.sum(1) + I * U * (np.abs(dh) * act[r] * np.abs(u[r])).sum(1)
        err = np.abs(dprob[r] - ref["dprob_perm"][r])
        assert np.all(err <= tol + 1e-30), f"{what} dprob: {(err / (tol + 1e-30)).max():.2f} times the tolerance"
        edz = np.concatenate([(edh + 20 * U * np.abs(dh)) * fg[r], (edh + 20 * U * np.abs(dh)) * fu[r]], 1)
        dz = np.abs(ref["dz"][r])
        edz = edz + HALF * (dz + edz)
        eh = (HALF + 20 * U) * np.abs(ref["h"][r])

        def close(a, b, prod, mags, terms, name):
            t = HALF * np.abs(b) + (1 + HALF) * (prod + terms * U * mags) + 1e-30
            q = np.abs(a - b) / t
            assert np.all(q <= 1), f"{what} {name} of expert {e}: {q.max():.2f} times the tolerance"
            if np.linalg.norm(b) > 0:  # independent roundings of what goes in and of the result
                assert np.linalg.norm(a - b) <= 2 * HALF * np.linalg.norm(b), f"{what} {name} of expert {e} (norm)"

        close(dx[r], ref["dx_perm"][r], edz @ np.abs(w1[e]), (dz + edz) @ np.abs(w1[e]), 2 * I, "dx")
        close(dw1[e], ref["dw_gate_up"][e], edz.T @ np.abs(xv[r]), (dz + edz).T @ np.abs(xv[r]), m, "dw1")
        close(dw2[e], ref["dw_down"][e], np.abs(dy[r]).T @ eh, np.abs(dy[r]).T @ np.abs(ref["h"][r]), m, "dw2")


# an expert of many row tiles (the last ones whole and ragged), one row, idle ones first, in the
# middle and last; K of few and of many steps (above 512 the tiles are split along K, but where they
# fill more than half of the card, as [1000] does); H wider and narrower than I
CASES = [([600], 256, 256, 0), ([1], 256, 256, 0), ([0, 3, 0, 0, 257, 0], 256, 512, 0), ([256, 255, 1], 512, 256, 5),
         ([0, 0], 256, 256, 4), ([40, 300, 17, 0], 1024, 256, 0), ([513, 64], 768, 768, 31), ([64] * 16, 256, 256, 0),
         ([700], 512, 1024, 0), ([1000], 768, 4352, 0), ([5, 0, 9], 2048, 768, 0), ([1, 0, 3, 2] * 64, 256, 256, 3)]


@pytest.mark.parametrize("counts,H,I,behind", CASES)
def test_forward_and_backward(moe, counts, H, I, behind):
    print(f"ckpt8 rows {counts} H={H} I={I} behind={behind}", flush=True)
    c = Case(counts, H, I, seed=H + I + sum(counts), behind=behind)
    zc, zs = _forward_check(moe, c)
    tc, ts = moe.mxfp8_quantize(c.tokens)
    xv = oracle.mxfp8_dequantize(host(tc), host(ts))[c.src.cpu().numpy()]
    got = moe.moe_grouped_mlp_bwd_ckpt8(c.dy, tc, zc, zs, c.prob, c.w1, c.w2, c.offsets, x_scale=ts, src_token=c.src)
    _backward_check(moe, c, zc, zs, got, xv, "tokens in 8 bits")
    # the same rows in expert order, and as bf16 (the values are exact in bf16): the same bits
    rc, rs = tc[c.src.long()].contiguous(), ts[c.src.long()].contiguous()
    for kw in (dict(x=rc, x_scale=rs), dict(x=moe.mxfp8_dequantize(rc, rs))):
        again = moe.moe_grouped_mlp_bwd_ckpt8(c.dy, kw.pop("x"), zc, zs, c.prob, c.w1, c.w2, c.offsets, **kw)
        for a, b, n in zip(again, got, ("dx", "dw1", "dw2", "dprob")):
            rows = c.used if n in ("dx", "dprob") else None
            assert torch.equal(a[:rows], b[:rows]), n


def test_weights_in_separate_tensors_and_given_outputs(moe):
    c = Case([5, 0, 300], 256, 256, seed=9)
    y, zc, zs = moe.moe_grouped_mlp_fwd_ckpt8(c.x, c.w1, c.w2, c.offsets, c.prob)
    out, ws = torch.empty_like(y), torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    w1, w2 = [w.clone() for w in c.w1], [w.clone() for w in c.w2]
    y2, zc2, zs2 = moe.moe_grouped_mlp_fwd_ckpt8(c.x, w1, w2, c.offsets, c.prob, out=out, workspace=ws)
    assert y2 is out and torch.equal(y, y2) and torch.equal(zc, zc2) and torch.equal(zs, zs2)
    a = moe.moe_grouped_mlp_bwd_ckpt8(c.dy, c.x, zc, zs, c.prob, c.w1, c.w2, c.offsets)
    outs = [torch.full_like(t, float("nan")) for t in a[:3]]
    b = moe.moe_grouped_mlp_bwd_ckpt8(c.dy, c.x, zc, zs, c.prob, w1, w2, c.offsets, dx_perm=outs[0], dw_gate_up=outs[1],
                                      dw_down=outs[2], workspace=torch.empty(1 << 30, dtype=torch.uint8, device="cuda"))
    for i, (s, t) in enumerate(zip(a, b)):
        assert torch.equal(s, t) and (i == 3 or t is outs[i])


def _raw(moe, c, zc, zs, y, dx, dprob, tc, ts):
    """Both entry points through the C ABI, on outputs that the caller filled."""
    from grouped_expert_gemm_amd import _lib
    L, s = _lib.lib(), torch.cuda.current_stream().cuda_stream
    tab = lambda w: (ctypes.c_void_p * c.E)(*[w[e].data_ptr() for e in range(c.E)])
    d = _lib.MlpDesc(c.E, c.H, c.I, 1, 1, 1, 0)
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    P = lambda t: t.data_ptr()
    assert L.moe_grouped_mlp_fwd_ckpt8(ctypes.byref(d), c.R, P(c.x), tab(c.w1), tab(c.w2), P(c.offsets), P(c.prob), P(y), P(zc),
                                       P(zs), P(ws), ws.numel(), s) == 0
    d.act = _lib.MOE_MXFP8
    dw1, dw2 = torch.empty_like(c.w1), torch.empty_like(c.w2)
    assert L.moe_grouped_mlp_bwd_ckpt8(ctypes.byref(d), c.R, P(c.dy), P(tc), P(ts), c.T, P(c.src), P(zc), P(zs), P(c.prob),
                                       tab(c.w1), tab(c.w2), P(c.offsets), P(dx), tab(dw1), tab(dw2), P(dprob), P(ws),
                                       ws.numel(), s) == 0
    return dw1, dw2


@pytest.mark.parametrize("counts,behind", [([600], 90), ([3, 0, 70], 41), ([0, 0], 33)])
def test_rows_behind_the_last_expert(moe, counts, behind):
    """Left as they were in every output; a token index there is not looked at, nor their NaN operands."""
    print(f"ckpt8 rows behind {counts} {behind}", flush=True)
    c = Case(counts, 256, 256, seed=21, behind=behind)
    c.x[c.used:], c.dy[c.used:], c.prob[c.used:] = float("nan"), float("nan"), float("nan")
    c.src[c.used:] = 2 ** 31 - 1
    tc, ts = moe.mxfp8_quantize(c.tokens)
    y = torch.full((c.R, c.H), 3.0, dtype=torch.bfloat16, device="cuda")
    dx, dprob = torch.full_like(y, 5.0), torch.full((c.R,), 6.0, device="cuda")
    zc = torch.full((c.R, 2 * c.I), 77, dtype=torch.uint8, device="cuda")
    zs = torch.full((c.R, c.I // 16), 78, dtype=torch.uint8, device="cuda")
    dw1, dw2 = _raw(moe, c, zc, zs, y, dx, dprob, tc, ts)
    n = c.used
    for t, v in ((y, 3.0), (dx, 5.0), (dprob, 6.0), (zc, 77), (zs, 78)):
        assert bool((t[n:] == v).all())
        assert n == 0 or not bool(torch.isnan(t[:n].float()).any())
    assert not bool(torch.isnan(dw1.float()).any()) and not bool(torch.isnan(dw2.float()).any())
    if n:
        want = moe.moe_grouped_mlp_bwd_ckpt8(c.dy, tc, zc, zs, c.prob, c.w1, c.w2, c.offsets, x_scale=ts, src_token=c.src)
        for a, b in zip((dx[:n], dw1, dw2, dprob[:n]), want):
            assert torch.equal(a, b[:n] if a.shape[0] == n else b)
    else:
        assert not dw1.any() and not dw2.any()


def test_tokens_out_of_range_read_as_zeros(moe):
    c = Case([30, 34], 256, 256, seed=5)
    _, zc, zs = moe.moe_grouped_mlp_fwd_ckpt8(c.x, c.w1, c.w2, c.offsets, c.prob)
    tc, ts = moe.mxfp8_quantize(c.tokens)
    lost = c.src.clone()
    lost[::5], lost[1::7] = -1, c.T
    got = moe.moe_grouped_mlp_bwd_ckpt8(c.dy, tc, zc, zs, c.prob, c.w1, c.w2, c.offsets, x_scale=ts, src_token=lost)
    xv = moe.mxfp8_dequantize(tc, ts)[c.src.long()]
    xv[::5], xv[1::7] = 0, 0
    want = moe.moe_grouped_mlp_bwd_ckpt8(c.dy, xv, zc, zs, c.prob, c.w1, c.w2, c.offsets)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_rows(moe):
    c = Case([0, 0, 0], 256, 256, seed=5)
    y, zc, zs = moe.moe_grouped_mlp_fwd_ckpt8(c.x, c.w1, c.w2, c.offsets, c.prob)
    assert y.shape == (0, 256) and zc.shape == (0, 512) and zs.shape == (0, 16)
    dx, dw1, dw2, dprob = moe.moe_grouped_mlp_bwd_ckpt8(c.dy, c.x, zc, zs, c.prob, c.w1, c.w2, c.offsets)
    assert dx.shape == (0, 256) and dprob.shape == (0,) and not dw1.any() and not dw2.any()


@pytest.mark.parametrize("counts", [[600], [20, 0, 9, 0]])
def test_values_that_are_not_finite(moe, counts):
    """A row whose z has an infinity or a NaN: blocks marked by the NaN scale, its gradients and its
    expert's weight gradients NaN; other rows and experts untouched."""
    c = Case(counts, 256, 256, seed=31)
    clean = moe.moe_grouped_mlp_fwd_ckpt8(c.x, c.w1, c.w2, c.offsets, c.prob)
    grads = moe.moe_grouped_mlp_bwd_ckpt8(c.dy, c.x, *clean[1:], c.prob, c.w1, c.w2, c.offsets)
    x = c.x.clone()
    x[4, 7] = float("inf")
    x[5, 9] = float("nan")
    y, zc, zs = moe.moe_grouped_mlp_fwd_ckpt8(x, c.w1, c.w2, c.offsets, c.prob)
    assert bool((zs[4:6] == 255).all()) and not bool(zc[4:6].any())
    keep = torch.ones(c.R, dtype=torch.bool, device="cuda")
    keep[4:6] = False
    assert torch.equal(zc[keep], clean[1][keep]) and torch.equal(zs[keep], clean[2][keep]) and torch.equal(y[keep], clean[0][keep])
    dx, dw1, dw2, dprob = moe.moe_grouped_mlp_bwd_ckpt8(c.dy, c.x, zc, zs, c.prob, c.w1, c.w2, c.offsets)
    assert bool(torch.isnan(dx[4:6]).all()) and bool(torch.isnan(dprob[4:6]).all())
    assert torch.equal(dx[keep], grads[0][keep]) and torch.equal(dprob[keep], grads[3][keep])
    assert bool(torch.isnan(dw1[0]).all()) and bool(torch.isnan(dw2[0]).all())
    for e in range(1, c.E):
        assert torch.equal(dw1[e], grads[1][e]) and torch.equal(dw2[e], grads[2][e])


def test_large_activations_saturate_the_gate(moe):
    """Gates far on both sides of zero, up to where e^-g overflows: silu, its slope and the codes stay finite."""
    c = Case([64, 40], 256, 256, seed=41)
    c.x *= 300.0
    zc, zs = _forward_check(moe, c)
    got = moe.moe_grouped_mlp_bwd_ckpt8(c.dy, c.x, zc, zs, c.prob, c.w1, c.w2, c.offsets)
    _backward_check(moe, c, zc, zs, got, host(c.x), "large activations")


def test_bad_offsets_stay_inside(moe):
    """Offsets that decrease or pass R are made nondecreasing inside [0, R]: the call ends and what lies past
    the tensors is untouched."""
    c = Case([100, 30], 256, 256, seed=6, behind=20)
    c.offsets[1], c.offsets[2] = 130, 4000
    zc = torch.full((c.R + 8, 2 * c.I), 77, dtype=torch.uint8, device="cuda")
    zs = torch.full((c.R + 8, c.I // 16), 78, dtype=torch.uint8, device="cuda")
    y = torch.full((c.R + 8, c.H), 3.0, dtype=torch.bfloat16, device="cuda")
    dx, dprob = torch.full_like(y, 5.0), torch.full((c.R + 8,), 6.0, device="cuda")
    tc, ts = moe.mxfp8_quantize(c.tokens)
    for e1 in (130, 4000, -5):
        c.offsets[1] = e1
        _raw(moe, c, zc, zs, y, dx, dprob, tc, ts)
        torch.cuda.synchronize()
        for t, v in ((y, 3.0), (dx, 5.0), (dprob, 6.0), (zc, 77), (zs, 78)):
            assert bool((t[c.R:] == v).all())


def test_refusals(moe):
    c = Case([20, 30], 256, 256, seed=3)
    _, zc, zs = moe.moe_grouped_mlp_fwd_ckpt8(c.x, c.w1, c.w2, c.offsets, c.prob)
    tc, ts = moe.mxfp8_quantize(c.tokens)
    fwd = dict(x_perm=c.x, w_gate_up=c.w1, w_down=c.w2, offsets=c.offsets, prob_perm=c.prob)
    for kw in (dict(x_perm=c.x.float()), dict(w_gate_up=c.w1.float()), dict(w_down=c.w2[:1]), dict(w_down=c.w1),
               dict(offsets=c.offsets.long()), dict(offsets=c.offsets[:2].contiguous()), dict(prob_perm=c.prob.double()),
               dict(prob_perm=c.prob[:3].contiguous()), dict(out=c.x.float()), dict(x_perm=c.x.t())):
        with pytest.raises(ValueError):
            moe.moe_grouped_mlp_fwd_ckpt8(**{**fwd, **kw})
    bwd = dict(dy_perm=c.dy, x=tc, z_codes=zc, z_scales=zs, prob_perm=c.prob, w_gate_up=c.w1, w_down=c.w2, offsets=c.offsets,
               x_scale=ts, src_token=c.src)
    for kw in (dict(dy_perm=c.dy.float()), dict(x=c.x), dict(x=c.x.float(), x_scale=None, src_token=None), dict(x_scale=None),
               dict(src_token=None), dict(src_token=c.src.long()), dict(src_token=c.src[:4].contiguous()),
               dict(z_codes=zc[:, :256].contiguous()), dict(z_scales=zs[:, :8].contiguous()), dict(z_codes=zc.int()),
               dict(dx_perm=c.dy.float()), dict(dw_gate_up=c.w2), dict(dw_down=c.w2.float()), dict(x=tc[:, :128].contiguous())):
        with pytest.raises(ValueError):
            moe.moe_grouped_mlp_bwd_ckpt8(**{**bwd, **kw})
    narrow = Case([20], 256, 128, seed=3)
    with pytest.raises(moe.MoeError, match="I % 256"):
        moe.moe_grouped_mlp_fwd_ckpt8(narrow.x, narrow.w1, narrow.w2, narrow.offsets, narrow.prob)
