"""MoE expert feed-forward hot path on AMD MI355X (gfx950): Python binding.

Thin argument marshalling over the C ABI of include/moe.h: every step runs in
the HIP kernels of libmoe.so; torch only provides device memory and the
current stream. The functions carry the C entry points' names.

Path (per "Efficient MoE Training for Biological Foundation Models",
Challenges 1-3): moe_route_topk -> moe_permute -> moe_grouped_mlp_fwd
(gate_up grouped GEMM + ScaledSwiGLU, down grouped GEMM) ->
moe_unpermute_combine; moe_grouped_mlp_bwd for the backward; mxfp8_quantize
for MXFP8 block quantisation. Around it: moe_pre_norm before the router,
moe_balance_loss on its logits, moe_post_norm in the place of
moe_unpermute_combine (combine, norm, gate, residual), each with its backward,
and MXFP4 experts for serving (mxfp4_quantize, compute="mxfp4").
Activations in 8 bits: moe_add_norm_mxfp8 (combine, residual, norm, MXFP8 rows),
mxfp8_dequantize, and moe_grouped_mlp_fwd_ckpt8 / moe_grouped_mlp_bwd_ckpt8, the
bf16 grouped MLP whose backward works from MXFP8 checkpoints.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from ._lib import MOE_BF16, MOE_F32, MOE_FP8, MOE_MXFP4, MOE_MXFP8, MlpDesc, MoeError, check, lib, ptr_table

__all__ = [
    "moe_route_topk", "moe_router_logits", "moe_route_topk_bwd", "moe_router_bwd", "moe_balance_loss",
    "moe_balance_loss_bwd", "moe_pre_norm", "moe_pre_norm_bwd", "moe_post_norm", "moe_post_norm_bwd",
    "moe_permute", "moe_unpermute_combine", "mxfp8_quantize", "mxfp4_quantize", "mxfp4_dequantize",
    "moe_grouped_linear_mxfp4", "moe_add_norm_mxfp8", "mxfp8_dequantize", "moe_grouped_mlp_fwd_ckpt8",
    "moe_grouped_mlp_bwd_ckpt8",
    "fp8_tensor_quantize", "mxfp8_quantize_colwise", "fp8_tensor_quantize_colwise", "mxfp8_pack_weight_bwd",
    "fp8_tensor_pack_weight_bwd", "mxfp8_quantize_weights", "fp8_tensor_quantize_weights",
    "moe_grouped_mlp_fwd", "moe_grouped_mlp_bwd", "moe_grouped_linear", "moe_grouped_gate_up_swiglu", "gemm_workspace",
    "workspace_size", "MoeError", "lib",
    "MOE_F32", "MOE_BF16", "MOE_MXFP8", "MOE_FP8", "MOE_MXFP4",
]

_DT = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.uint8: MOE_MXFP8}


def _stream(device=None):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _p(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _need_cuda(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("tensors must live on the GPU")
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")


def _need(fn, ref, *ts):
    """Every given tensor on ref's GPU and contiguous."""
    dev = ref.get_device()   # -1 on the CPU
    for t in (ref, *ts):
        if t is not None:
            if t.get_device() != dev or dev < 0:
                raise ValueError(f"{fn}: tensors must live on one GPU")
            if not t.is_contiguous():
                raise ValueError(f"{fn}: tensors must be contiguous")


def _a(t):
    """A tensor's address for a pointer argument (None: NULL)."""
    return t.data_ptr() if t is not None else None


def _launch(fn, t, *args):
    """Call entry point fn (its last argument, the stream, added) with t's GPU as the current device."""
    L = lib()
    dev = t.get_device()
    stream = torch._C._cuda_getCurrentRawStream(dev)  # torch.cuda.current_stream(dev).cuda_stream, 2 us faster
    if torch.cuda.current_device() == dev:
        status = getattr(L, fn)(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = getattr(L, fn)(*args, stream)
    if status:
        check(fn.removesuffix("_tables"), status)


def _workspace(nbytes, device):
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def workspace_size(op, desc=None, R=0, T=0, E=1, k=1):
    n = ctypes.c_size_t(0)
    check("moe_workspace_size", lib().moe_workspace_size(op, ctypes.byref(desc) if desc is not None else None,
                                                         R, T, E, k, ctypes.byref(n)))
    return n.value


@functools.lru_cache(maxsize=1024)
def _size(op, desc=None, R=0, T=0, E=1, k=1):
    """workspace_size of the fields of an MlpDesc: a function of its numbers alone."""
    return workspace_size(op, MlpDesc(*desc) if desc else None, R, T, E, k)


def moe_route_topk(logits: torch.Tensor, k: int, renormalize: bool = True):
    """logits [T, E] float32 -> (topk_idx int32 [T, k], topk_prob float32 [T, k])."""
    _need_cuda(logits)
    T, E = logits.shape
    idx = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    prob = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    check("moe_route_topk", lib().moe_route_topk(_p(logits), T, E, k, int(renormalize), _p(idx), _p(prob),
                                                 _stream(logits.device)))
    return idx, prob


def moe_router_logits(x: torch.Tensor, w_router: torch.Tensor) -> torch.Tensor:
    """x [T, H] bf16, w_router [E, H] bf16 -> logits [T, E] float32."""
    _need_cuda(x, w_router)
    T, H = x.shape
    E = w_router.shape[0]
    if x.dtype != torch.bfloat16 or w_router.dtype != torch.bfloat16 or w_router.shape[1] != H:
        raise ValueError("moe_router_logits: x [T, H] and w_router [E, H] must be bfloat16")
    logits = torch.empty((T, E), dtype=torch.float32, device=x.device)
    check("moe_router_logits", lib().moe_router_logits(_p(x), _p(w_router), T, H, E, _p(logits),
                                                       _stream(x.device)))
    return logits


def moe_route_topk_bwd(topk_idx: torch.Tensor, topk_prob: torch.Tensor, d_topk_prob: torch.Tensor, E: int,
                       renormalize: bool = True, logits: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of moe_route_topk's probabilities -> d_logits [T, E] float32
    (``logits`` is needed only without renormalisation)."""
    _need_cuda(topk_idx, topk_prob, d_topk_prob, logits)
    T, k = topk_idx.shape
    d = torch.empty((T, E), dtype=torch.float32, device=topk_idx.device)
    check("moe_route_topk_bwd", lib().moe_route_topk_bwd(_p(logits), _p(topk_idx), _p(topk_prob), _p(d_topk_prob),
                                                         T, E, k, int(renormalize), _p(d),
                                                         _stream(topk_idx.device)))
    return d


def moe_router_bwd(x: torch.Tensor, w_router: torch.Tensor, d_logits: torch.Tensor,
                   dx_in: torch.Tensor | None = None, dx: torch.Tensor | None = None):
    """Backward of moe_router_logits -> (dx [T, H] bf16 = dx_in + d_logits w_router,
    dw_router [E, H] float32 = d_logits^T x)."""
    _need_cuda(x, w_router, d_logits, dx_in, dx)
    T, H = x.shape
    E = w_router.shape[0]
    if dx is None:
        dx = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    dw = torch.empty((E, H), dtype=torch.float32, device=x.device)
    desc = MlpDesc(E, H, 1, 0, MOE_BF16, MOE_BF16, 0)
    ws = _workspace(workspace_size(_lib.MOE_OP_ROUTER_BWD, desc, 0, T), x.device)
    check("moe_router_bwd", lib().moe_router_bwd(_p(x), _p(w_router), _p(d_logits), _p(dx_in), T, H, E, _p(dx),
                                                 _p(dw), _p(ws), ws.numel(), _stream(x.device)))
    return dx, dw


def _seq_len(fn, T, seq_len):
    L = seq_len if seq_len is not None else max(T, 1)
    if L < 1 or T % L:
        raise ValueError(f"{fn}: seq_len must divide the number of tokens")
    return L


def _check_mask(fn, mask, T):
    if mask is not None and (mask.dtype not in (torch.uint8, torch.bool) or mask.shape != (T,)):
        raise ValueError(f"{fn}: mask must be bool or uint8 [T]")


def moe_balance_loss(logits: torch.Tensor, topk_idx: torch.Tensor, balance_coef: float, z_coef: float = 0.0,
                     seq_len: int | None = None, mask: torch.Tensor | None = None):
    """Load-balance loss (with z-loss) of router logits [T, E] float32 routed to topk_idx [T, k] int32.

    Returns (loss [3] float32: loss, mean balance term, mean z term; counts [T / seq_len, E] int32;
    tokens [T / seq_len + 1] int32: counted tokens per sequence, then the sequences that have any).
    seq_len: tokens per sequence (default: one loss over all T); mask [T]: 0 leaves a token out."""
    _need("moe_balance_loss", logits, topk_idx, mask)
    T, E = logits.shape
    if logits.dtype != torch.float32 or topk_idx.dtype != torch.int32 or topk_idx.shape[0] != T:
        raise ValueError("moe_balance_loss: logits [T, E] must be float32 and topk_idx [T, k] int32")
    _check_mask("moe_balance_loss", mask, T)
    L = _seq_len("moe_balance_loss", T, seq_len)
    dev = logits.device
    counts = torch.empty((T // L, E), dtype=torch.int32, device=dev)
    tokens = torch.empty(T // L + 1, dtype=torch.int32, device=dev)
    loss = torch.empty(3, dtype=torch.float32, device=dev)
    need = _size(_lib.MOE_OP_BALANCE_LOSS, None, L, T, E)
    ws = _workspace(need, dev) if need else None
    _launch("moe_balance_loss", logits, _a(logits), _a(topk_idx), _a(mask), T, E, topk_idx.shape[1], L, balance_coef,
            z_coef, _a(counts), _a(tokens), _a(loss), _a(ws), need)
    return loss, counts, tokens


def moe_balance_loss_bwd(logits: torch.Tensor, counts: torch.Tensor, tokens: torch.Tensor, k: int,
                         balance_coef: float, z_coef: float = 0.0, seq_len: int | None = None,
                         mask: torch.Tensor | None = None, d_loss: torch.Tensor | None = None,
                         d_logits_in: torch.Tensor | None = None, d_logits: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of moe_balance_loss's loss[0] in the logits, times d_loss ([1] float32, default 1), plus
    d_logits_in ([T, E] float32, default 0): d_logits [T, E] float32 (may be d_logits_in itself)."""
    _need("moe_balance_loss_bwd", logits, counts, tokens, mask, d_loss, d_logits_in, d_logits)
    T, E = logits.shape
    _check_mask("moe_balance_loss_bwd", mask, T)
    L = _seq_len("moe_balance_loss_bwd", T, seq_len)
    for t, shape in ((d_logits_in, logits.shape), (d_logits, logits.shape)):
        if t is not None and (t.dtype != torch.float32 or t.shape != shape):
            raise ValueError("moe_balance_loss_bwd: d_logits_in and d_logits must be float32 [T, E]")
    if (logits.dtype != torch.float32 or counts.dtype != torch.int32 or counts.shape != (T // L, E)
            or tokens.dtype != torch.int32 or tokens.numel() != T // L + 1
            or (d_loss is not None and (d_loss.dtype != torch.float32 or d_loss.numel() != 1))):
        raise ValueError("moe_balance_loss_bwd: logits and d_loss must be float32, counts and tokens the forward's")
    if d_logits is None:
        d_logits = torch.empty_like(logits)
    _launch("moe_balance_loss_bwd", logits, _a(logits), _a(counts), _a(tokens), _a(mask), T, E, k, L,
            balance_coef, z_coef, _a(d_loss), _a(d_logits_in), _a(d_logits))
    return d_logits


def _norm_dtype(fn, x, *same):
    if x.dtype not in (torch.float32, torch.bfloat16) or x.dim() != 2:
        raise ValueError(f"{fn}: rows must be a 2-D float32 or bfloat16 tensor")
    for t in same:
        if t is not None and t.dtype != x.dtype:
            raise ValueError(f"{fn}: all tensors but rstd and the maps must share one dtype")
    return _DT[x.dtype]


def _gate_args(fn, gate, gate_group, T, H):
    """(kind, group) of a gate tensor: [T] per token, [G, H] one row for every gate_group tokens."""
    if gate is None:
        return _lib.MOE_GATE_NONE, 1
    if gate.dim() == 1:
        if gate.shape[0] != T:
            raise ValueError(f"{fn}: a gate per token must be [T]")
        return _lib.MOE_GATE_TOKEN, 1
    group = gate_group if gate_group is not None else max(1, -(-T // max(gate.shape[0], 1)))
    if gate.dim() != 2 or gate.shape[1] != H or group < 1 or (T > 0 and gate.shape[0] != -(-T // group)):
        raise ValueError(f"{fn}: a channel gate must be [ceil(T / gate_group), H]")
    return _lib.MOE_GATE_CHANNEL, group


def _check_rows(fn, row_id_map, T, k):
    if row_id_map is None:
        if k != 1:
            raise ValueError(f"{fn}: k > 1 needs row_id_map")
    elif row_id_map.dtype != torch.int32 or row_id_map.numel() != T * k:
        raise ValueError(f"{fn}: row_id_map must be int32 [T * k]")


def moe_pre_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, save_rstd: bool = False):
    """RMS norm of the rows of x [T, H] (bf16 or float32) with weight [H]: y, or (y, rstd [T]) with save_rstd."""
    _need("moe_pre_norm", x, weight)
    dt = _norm_dtype("moe_pre_norm", x, weight)
    T, H = x.shape
    if weight.shape != (H,):
        raise ValueError("moe_pre_norm: weight must be [H]")
    y = torch.empty_like(x)
    rstd = torch.empty(T, dtype=torch.float32, device=x.device) if save_rstd else None
    _launch("moe_pre_norm", x, _a(x), _a(weight), dt, T, H, eps, _a(y), _a(rstd))
    return (y, rstd) if save_rstd else y


def _norm_workspace(T, H, kind, group, dev):
    return _workspace(_size(_lib.MOE_OP_NORM_BWD, (1, H, 1, 0, 0, 0, 0), 0, T, kind, max(1, min(group, T))), dev)


def moe_pre_norm_bwd(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                     dx_in: torch.Tensor | None = None, dx_in_scale: float = 1.0, dx: torch.Tensor | None = None):
    """Backward of moe_pre_norm -> (dx [T, H] = dx_in_scale * dx_in + the norm's gradient, dweight [H] float32)."""
    _need("moe_pre_norm_bwd", x, dy, weight, rstd, dx_in, dx)
    dt = _norm_dtype("moe_pre_norm_bwd", x, dy, weight, dx_in, dx)
    T, H = x.shape
    if weight.shape != (H,) or rstd.dtype != torch.float32 or rstd.shape != (T,):
        raise ValueError("moe_pre_norm_bwd: weight must be [H] and rstd float32 [T]")
    for t in (dy, dx_in, dx):
        if t is not None and t.shape != x.shape:
            raise ValueError("moe_pre_norm_bwd: dy, dx_in and dx must have x's shape")
    if dx is None:
        dx = torch.empty_like(x)
    dw = torch.empty(H, dtype=torch.float32, device=x.device)
    ws = _norm_workspace(T, H, _lib.MOE_GATE_NONE, 1, x.device)
    _launch("moe_pre_norm_bwd", x, _a(dy), _a(x), _a(weight), _a(rstd), _a(dx_in), dx_in_scale, dt, T, H,
            _a(dx), _a(dw), _a(ws), ws.numel())
    return dx, dw


def moe_post_norm(y: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, row_id_map: torch.Tensor | None = None,
                  k: int = 1, gate: torch.Tensor | None = None, gate_group: int | None = None,
                  residual_scale: float = 1.0, eps: float = 1e-6, save_for_bwd: bool = False,
                  next_weight: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """out = residual_scale * x + gate * RMSNorm(c) * weight with c[t] the sum of token t's k rows of y
    (through row_id_map, as moe_unpermute_combine) or y[t] itself without a map.

    gate: None, [T] (per token) or [ceil(T / gate_group), H] (one row for every gate_group consecutive tokens;
    default: T over the gate's rows). Returns a dict with out, c and rstd with save_for_bwd, y_next
    (moe_pre_norm of out) with next_weight, and rstd_next with both. out may be x."""
    _need("moe_post_norm", x, y, weight, row_id_map, gate, next_weight, out)
    dt = _norm_dtype("moe_post_norm", x, y, weight, gate, next_weight, out)
    T, H = x.shape
    _check_rows("moe_post_norm", row_id_map, T, k)
    kind, group = _gate_args("moe_post_norm", gate, gate_group, T, H)
    if y.shape != (T * k, H) or weight.shape != (H,) or (next_weight is not None and next_weight.shape != (H,)):
        raise ValueError("moe_post_norm: y must be [T * k, H] and the weights [H]")
    if out is not None and out.shape != x.shape:
        raise ValueError("moe_post_norm: out must have x's shape")
    dev = x.device
    r = dict(out=out if out is not None else torch.empty_like(x))
    if save_for_bwd:
        r["c"] = torch.empty_like(x)
        r["rstd"] = torch.empty(T, dtype=torch.float32, device=dev)
    if next_weight is not None:
        r["y_next"] = torch.empty_like(x)
        if save_for_bwd:
            r["rstd_next"] = torch.empty(T, dtype=torch.float32, device=dev)
    _launch("moe_post_norm", x, _a(y), _a(row_id_map), k, _a(x), _a(weight), kind, _a(gate), group, residual_scale,
            _a(next_weight), dt, T, H, eps, _a(r["out"]), _a(r.get("c")), _a(r.get("rstd")), _a(r.get("y_next")),
            _a(r.get("rstd_next")))
    return r


def moe_post_norm_bwd(dout: torch.Tensor, c: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor,
                      row_id_map: torch.Tensor | None = None, k: int = 1, gate: torch.Tensor | None = None,
                      gate_group: int | None = None, dy: torch.Tensor | None = None):
    """Backward of moe_post_norm: a dict with dy [T * k, H] (the gradient of every row, in y's order; rows no slot
    points at are left as they were), dweight [H] float32 and dgate (float32, the gate's shape, with a gate)."""
    _need("moe_post_norm_bwd", dout, c, rstd, weight, row_id_map, gate, dy)
    dt = _norm_dtype("moe_post_norm_bwd", dout, c, weight, gate, dy)
    T, H = dout.shape
    _check_rows("moe_post_norm_bwd", row_id_map, T, k)
    kind, group = _gate_args("moe_post_norm_bwd", gate, gate_group, T, H)
    if c.shape != dout.shape or weight.shape != (H,) or rstd.dtype != torch.float32 or rstd.shape != (T,):
        raise ValueError("moe_post_norm_bwd: c must have dout's shape, weight [H] and rstd float32 [T]")
    if dy is None:
        dy = torch.empty((T * k, H), dtype=dout.dtype, device=dout.device)
    elif dy.shape != (T * k, H):
        raise ValueError("moe_post_norm_bwd: dy must be [T * k, H]")
    dev = dout.device
    dw = torch.empty(H, dtype=torch.float32, device=dev)
    dgate = None
    if gate is not None:
        dgate = (torch.empty if T > 0 else torch.zeros)(gate.shape, dtype=torch.float32, device=dev)
    ws = _norm_workspace(T, H, kind, group, dev)
    _launch("moe_post_norm_bwd", dout, _a(dout), _a(c), _a(rstd), _a(weight), kind, _a(gate), group, _a(row_id_map), k,
            dt, T, H, _a(dy), _a(dw), _a(dgate), _a(ws), ws.numel())
    r = dict(dy=dy, dweight=dw)
    if gate is not None:
        r["dgate"] = dgate
    return r


def moe_add_norm_mxfp8(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                       row_id_map: torch.Tensor | None = None, k: int = 1, eps: float = 1e-6, with_y: bool = False,
                       save_for_bwd: bool = False, out: torch.Tensor | None = None):
    """s = residual + x (or, through row_id_map, residual + the sum of each token's k rows of x, as
    moe_unpermute_combine without weights), its RMS norm n = s * rstd * weight, and n's MXFP8 rows.

    x [T, H] or [T * k, H], residual [T, H], weight [H]: bf16 or float32, one dtype; H % 32 == 0. Returns a dict with
    codes uint8 [T, H], scales uint8 [T, H / 32], sum [T, H] (s as the norm read it; x itself where nothing is
    added and out is not given), y (n in x's dtype) with with_y, and rstd [T] with save_for_bwd. out: the sum's
    tensor, may be residual. Backward: moe_pre_norm_bwd(dy, sum, weight, rstd, dx_in=the gradient past the norm)."""
    fn = "moe_add_norm_mxfp8"
    _need(fn, x, weight, residual, row_id_map, out)
    dt = _norm_dtype(fn, x, weight, residual, out)
    if k < 1 or (row_id_map is not None and x.shape[0] % k):
        raise ValueError(f"{fn}: k must be positive and x [T * k, H]")
    T, H = x.shape[0] // k, x.shape[1]
    _check_rows(fn, row_id_map, T, k)
    if weight.shape != (H,):
        raise ValueError(f"{fn}: weight must be [H]")
    for t in (residual, out):
        if t is not None and t.shape != (T, H):
            raise ValueError(f"{fn}: residual and out must be [T, H]")
    added = out
    if added is None and residual is not None:
        added = torch.empty_like(residual)
    elif added is None and row_id_map is not None:
        added = x.new_empty((T, H))
    r = dict(sum=added if added is not None else x)
    rows = r["sum"]
    r["codes"] = torch.empty_like(rows, dtype=torch.uint8)
    r["scales"] = r["codes"].new_empty((T, H // 32))
    if with_y:
        r["y"] = torch.empty_like(rows)
    if save_for_bwd:
        r["rstd"] = torch.empty(T, dtype=torch.float32, device=x.device)
    _launch(fn, x, _a(x), _a(row_id_map), k, _a(residual), _a(weight), dt, T, H, eps, _a(added), _a(r.get("y")),
            _a(r.get("rstd")), _a(r["codes"]), _a(r["scales"]))
    return r


def moe_permute(x: torch.Tensor, topk_idx: torch.Tensor, topk_prob: torch.Tensor | None, E: int,
                x_scale: torch.Tensor | None = None, row_id_map: torch.Tensor | None = None):
    """Group the (token, slot) pairs by expert.

    Returns a dict with x_perm [R, H], x_perm_scale (MXFP8 and MXFP4 only), prob_perm [R],
    split_sizes [E], offsets [E+1], row_id_map [T*k], src_token [R].
    uint8 codes x [T, B] come with x_scale, a byte per 32 values: MXFP4 (two values a byte)
    where x_scale is [T, B / 16], else MXFP8 with T * B / 32 bytes of scales.
    With ``row_id_map`` given, only x is gathered with that map (topk_idx gives k).
    """
    _need_cuda(x, topk_idx, topk_prob, x_scale, row_id_map)
    T, H = x.shape
    k = topk_idx.shape[1]
    R = T * k
    dt = _DT[x.dtype]
    dev = x.device
    x_perm = torch.empty((R, H), dtype=x.dtype, device=dev)
    if dt == MOE_MXFP8 and x_scale is not None:
        if x_scale.shape == (T, H // 16):
            dt, H = MOE_MXFP4, 2 * H   # two codes a byte
        elif x_scale.numel() < T * (H // 32):
            raise ValueError("moe_permute: x_scale must be [T, H/32] (MXFP8) or, of x's bytes a row, [T, bytes/16] (MXFP4)")
    xps = torch.empty((R, H // 32), dtype=torch.uint8, device=dev) if dt in (MOE_MXFP8, MOE_MXFP4) else None
    if row_id_map is not None:
        check("moe_permute", lib().moe_permute(_p(x), _p(x_scale), dt, T, H, E, k, None, None, 1, _p(x_perm),
                                               _p(xps), None, None, None, _p(row_id_map), None, None, 0,
                                               _stream(dev)))
        return dict(x_perm=x_perm, x_perm_scale=xps)
    prob_perm = torch.empty(R, dtype=torch.float32, device=dev) if topk_prob is not None else None
    split = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    rmap = torch.empty(R, dtype=torch.int32, device=dev)
    src = torch.empty(R, dtype=torch.int32, device=dev)
    ws = _workspace(workspace_size(_lib.MOE_OP_PERMUTE, None, 0, T, E, k), dev)
    check("moe_permute", lib().moe_permute(_p(x), _p(x_scale), dt, T, H, E, k, _p(topk_idx), _p(topk_prob), 0,
                                           _p(x_perm), _p(xps), _p(prob_perm), _p(split), _p(offsets), _p(rmap),
                                           _p(src), _p(ws), ws.numel(), _stream(dev)))
    return dict(x_perm=x_perm, x_perm_scale=xps, prob_perm=prob_perm, split_sizes=split, offsets=offsets,
                row_id_map=rmap, src_token=src)


def moe_unpermute_combine(y_perm: torch.Tensor, row_id_map: torch.Tensor, T: int, k: int,
                          weights: torch.Tensor | None = None):
    """out[t] = sum_j w[t, j] * y_perm[row_id_map[t*k + j]] (w = 1 without weights)."""
    _need_cuda(y_perm, row_id_map, weights)
    H = y_perm.shape[1]
    out = torch.empty((T, H), dtype=y_perm.dtype, device=y_perm.device)
    check("moe_unpermute_combine", lib().moe_unpermute_combine(_p(y_perm), _DT[y_perm.dtype], _p(row_id_map),
                                                               _p(weights), T, H, k, _p(out),
                                                               _stream(y_perm.device)))
    return out


def mxfp8_quantize(x: torch.Tensor):
    """bf16 [rows, cols] -> (E4M3 codes uint8 [rows, cols], E8M0 scales uint8 [rows, cols/32])."""
    _need_cuda(x)
    if x.dtype != torch.bfloat16:
        raise ValueError("mxfp8_quantize takes bfloat16")
    x2 = x.reshape(-1, x.shape[-1])
    rows, cols = x2.shape
    codes = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    scales = torch.empty((rows, cols // 32), dtype=torch.uint8, device=x.device)
    check("mxfp8_quantize", lib().mxfp8_quantize(_p(x2), rows, cols, _p(codes), _p(scales), _stream(x.device)))
    return codes.reshape(x.shape), scales.reshape(*x.shape[:-1], cols // 32)


def mxfp8_dequantize(codes: torch.Tensor, scales: torch.Tensor, src_row: torch.Tensor | None = None,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    """MXFP8 codes [..., cols] and scales [..., cols/32] -> their values, bf16 [..., cols].

    src_row int32 [rows] (codes 2-D): out[r] = the values of row src_row[r], bf16 [rows, cols]; rows whose
    index is out of range are zeros, or, where out is given, left as they were."""
    fn = "mxfp8_dequantize"
    _need(fn, codes, scales, src_row, out)
    shape = codes.shape
    if codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or not shape or scales.dim() != len(shape) \
            or scales.shape[:-1] != shape[:-1] or scales.shape[-1] != shape[-1] // 32:
        raise ValueError(f"{fn}: codes must be uint8 [..., cols] and scales uint8 [..., cols/32]")
    cols = shape[-1]
    src_rows = codes.numel() // cols if cols else 0
    if src_row is not None:
        if len(shape) != 2 or src_row.dtype != torch.int32 or src_row.dim() != 1:
            raise ValueError(f"{fn}: src_row must be int32 [rows], with 2-D codes")
        shape = (src_row.shape[0], cols)
    entry = fn
    if out is None:
        out = codes.new_empty(shape, dtype=torch.bfloat16)
        entry = fn if src_row is None else "mxfp8_dequantize_gather"
    elif out.dtype != torch.bfloat16 or out.shape != shape:
        raise ValueError(f"{fn}: out must be bfloat16 [rows, cols]")
    rows = src_rows if src_row is None else shape[0]
    _launch(entry, codes, _a(codes), _a(scales), src_rows, cols, _a(src_row), rows, _a(out))
    return out


def mxfp4_quantize(x: torch.Tensor):
    """bf16 [..., cols] -> (E2M1 codes uint8 [..., cols/2], two a byte, the even one in the low
    nibble; E8M0 scales uint8 [..., cols/32])."""
    _need("mxfp4_quantize", x)
    if x.dtype != torch.bfloat16 or x.dim() < 1:
        raise ValueError("mxfp4_quantize takes bfloat16")
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    codes = torch.empty((*x.shape[:-1], cols // 2), dtype=torch.uint8, device=x.device)
    scales = torch.empty((*x.shape[:-1], cols // 32), dtype=torch.uint8, device=x.device)
    _launch("mxfp4_quantize", x, _a(x), rows, cols, _a(codes), _a(scales))
    return codes, scales


def mxfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """MXFP4 codes [..., cols/2] and scales [..., cols/32] -> their values, bf16 [..., cols]."""
    _need("mxfp4_dequantize", codes, scales)
    if codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or scales.shape != (*codes.shape[:-1],
                                                                                     codes.shape[-1] // 16):
        raise ValueError("mxfp4_dequantize: codes must be uint8 [..., cols/2] and scales uint8 [..., cols/32]")
    cols = 2 * codes.shape[-1]
    rows = codes.numel() // codes.shape[-1] if cols else 0
    out = torch.empty((*codes.shape[:-1], cols), dtype=torch.bfloat16, device=codes.device)
    _launch("mxfp4_dequantize", codes, _a(codes), _a(scales), rows, cols, _a(out))
    return out


def fp8_tensor_quantize(x: torch.Tensor):
    """bf16 tensor -> (E4M3 codes uint8 of x's shape, float32 scale tensor of shape [1])."""
    _need_cuda(x)
    if x.dtype != torch.bfloat16:
        raise ValueError("fp8_tensor_quantize takes bfloat16")
    x = x.contiguous()
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    scale = torch.empty(1, dtype=torch.float32, device=x.device)
    check("fp8_tensor_quantize", lib().fp8_tensor_quantize(_p(x), x.numel(), _p(codes), _p(scale),
                                                           _stream(x.device)))
    return codes, scale


def mxfp8_quantize_colwise(x: torch.Tensor, offsets: torch.Tensor, pad: int = 32):
    """bf16 [R, C] with expert row offsets [E+1] -> (E4M3 codes [C, kcap], E8M0 scales
    [C, kcap/32], padded offsets kofs [E+1]) with kcap = R + E * (pad - 1) rounded up to
    128 (whole cache lines per output row): each expert's rows, zero-padded to a
    multiple of pad, quantised along the token axis as columns [kofs[e], kofs[e+1])."""
    _need_cuda(x, offsets)
    if x.dtype != torch.bfloat16:
        raise ValueError("mxfp8_quantize_colwise takes bfloat16")
    x = x.contiguous()
    R, C = x.shape
    E = offsets.numel() - 1
    kcap = (R + E * (pad - 1) + 127) // 128 * 128
    codes = torch.zeros((C, kcap), dtype=torch.uint8, device=x.device)
    scales = torch.zeros((C, kcap // 32), dtype=torch.uint8, device=x.device)
    kofs = torch.empty(E + 1, dtype=torch.int32, device=x.device)
    check("mxfp8_quantize_colwise", lib().mxfp8_quantize_colwise(_p(x), R, C, E, _p(offsets), pad, kcap, _p(codes),
                                                                 _p(scales), _p(kofs), _stream(x.device)))
    return codes, scales, kofs


def fp8_tensor_quantize_colwise(x: torch.Tensor, offsets: torch.Tensor, pad: int = 256):
    """bf16 [R, C] with expert row offsets [E+1] -> (E4M3 codes [C, kcap], float32 scale
    [1], padded offsets kofs [E+1]) with kcap = R + E * (pad - 1) rounded up to 128: the
    per-tensor FP8 codes of x, each expert's rows zero-padded to a multiple of pad and
    transposed to columns [kofs[e], kofs[e+1])."""
    _need_cuda(x, offsets)
    if x.dtype != torch.bfloat16:
        raise ValueError("fp8_tensor_quantize_colwise takes bfloat16")
    x = x.contiguous()
    R, C = x.shape
    E = offsets.numel() - 1
    kcap = (R + E * (pad - 1) + 127) // 128 * 128
    codes = torch.zeros((C, kcap), dtype=torch.uint8, device=x.device)
    scale = torch.empty(1, dtype=torch.float32, device=x.device)
    kofs = torch.empty(E + 1, dtype=torch.int32, device=x.device)
    check("fp8_tensor_quantize_colwise", lib().fp8_tensor_quantize_colwise(
        _p(x), R, C, E, _p(offsets), pad, kcap, _p(codes), _p(scale), _p(kofs), _stream(x.device)))
    return codes, scale, kofs


def fp8_tensor_pack_weight_bwd(w: torch.Tensor) -> torch.Tensor:
    """bf16 weight [rows, cols] -> packed per-tensor FP8 for moe_grouped_mlp_bwd (uint8,
    rows * cols + 4 bytes: the codes of w^T, then the float32 factor)."""
    _need_cuda(w)
    if w.dtype != torch.bfloat16 or w.dim() != 2:
        raise ValueError("fp8_tensor_pack_weight_bwd takes a 2-D bfloat16 weight")
    w = w.contiguous()
    rows, cols = w.shape
    packed = torch.empty(rows * cols + 16, dtype=torch.uint8, device=w.device)
    check("fp8_tensor_pack_weight_bwd", lib().fp8_tensor_pack_weight_bwd(_p(w), rows, cols, _p(packed),
                                                                         _stream(w.device)))
    return packed


def mxfp8_pack_weight_bwd(w: torch.Tensor) -> torch.Tensor:
    """bf16 weight [rows, cols] -> packed MXFP8 for moe_grouped_mlp_bwd (uint8, rows * cols
    * 33 / 32 bytes: the codes of w^T quantised along rows, then the step-major scales)."""
    _need_cuda(w)
    if w.dtype != torch.bfloat16 or w.dim() != 2:
        raise ValueError("mxfp8_pack_weight_bwd takes a 2-D bfloat16 weight")
    rows, cols = w.shape
    packed = torch.empty(rows * cols + rows * cols // 32, dtype=torch.uint8, device=w.device)
    check("mxfp8_pack_weight_bwd", lib().mxfp8_pack_weight_bwd(_p(w), rows, cols, _p(packed), _stream(w.device)))
    return packed


def _weight_stack(w, fn):
    _need_cuda(w)
    if w.dtype != torch.bfloat16 or w.dim() != 3:
        raise ValueError(f"{fn} takes bfloat16 weights [n, rows, cols]")
    return w.contiguous()


def mxfp8_quantize_weights(w: torch.Tensor):
    """bf16 weights [n, rows, cols] -> (E4M3 codes uint8 [n, rows, cols], E8M0 scales uint8
    [n, rows, cols/32], packed uint8 [n, rows * cols * 33 / 32]): for each weight the
    outputs of mxfp8_quantize and of mxfp8_pack_weight_bwd, from one read of it."""
    w = _weight_stack(w, "mxfp8_quantize_weights")
    n, rows, cols = w.shape
    codes = torch.empty((n, rows, cols), dtype=torch.uint8, device=w.device)
    scales = torch.empty((n, rows, cols // 32), dtype=torch.uint8, device=w.device)
    packed = torch.empty((n, rows * cols + rows * cols // 32), dtype=torch.uint8, device=w.device)
    tw, kw = _lib.ptr_table([w[i].data_ptr() for i in range(n)])
    tc, kc = _lib.ptr_table([codes[i].data_ptr() for i in range(n)])
    ts, ks = _lib.ptr_table([scales[i].data_ptr() for i in range(n)])
    tp, kp = _lib.ptr_table([packed[i].data_ptr() for i in range(n)])
    check("mxfp8_quantize_weights", lib().mxfp8_quantize_weights(n, tw, rows, cols, tc, ts, tp, _stream(w.device)))
    return codes, scales, packed


def fp8_tensor_quantize_weights(w: torch.Tensor):
    """bf16 weights [n, rows, cols] -> (E4M3 codes uint8 [n, rows, cols], float32 scales [n],
    packed uint8 [n, rows * cols + 16]): for each weight the outputs of
    fp8_tensor_quantize and of fp8_tensor_pack_weight_bwd (in the first rows * cols + 4
    bytes of its packed row), from one pass for the maxima and one for the codes."""
    w = _weight_stack(w, "fp8_tensor_quantize_weights")
    n, rows, cols = w.shape
    codes = torch.empty((n, rows, cols), dtype=torch.uint8, device=w.device)
    scale = torch.empty(n, dtype=torch.float32, device=w.device)
    packed = torch.empty((n, rows * cols + 16), dtype=torch.uint8, device=w.device)
    tw, kw = _lib.ptr_table([w[i].data_ptr() for i in range(n)])
    tc, kc = _lib.ptr_table([codes[i].data_ptr() for i in range(n)])
    tp, kp = _lib.ptr_table([packed[i].data_ptr() for i in range(n)])
    check("fp8_tensor_quantize_weights", lib().fp8_tensor_quantize_weights(n, tw, rows, cols, tc, _p(scale), tp,
                                                                           _stream(w.device)))
    return codes, scale, packed


def _experts(w):
    """A [E, ...] tensor or a list of per-expert tensors -> list of per-expert tensors."""
    if isinstance(w, torch.Tensor):
        return [w[e] for e in range(w.shape[0])]
    return list(w)


def _weight_table(fn, w, dev):
    """Per-expert weights, one tensor [E, ...] or a list -> (pointer table, E, shape, dtype). One
    tensor's pointers are a stride apart, so a call does not touch E slices."""
    if isinstance(w, torch.Tensor):
        if w.get_device() != dev or not w.is_contiguous() or w.numel() == 0:
            raise ValueError(f"{fn}: weights must be contiguous, not empty, and live on the rows' GPU")
        E, *shape = w.shape
        table = (ctypes.c_void_p * E)()
        lib().moe_pointer_table(w.data_ptr(), w.stride(0) * w.element_size(), E, table)
        return table, E, tuple(shape), w.dtype
    w = list(w)
    if not w:
        raise ValueError(f"{fn}: no weights")
    for t in w:
        if t.get_device() != dev or not t.is_contiguous() or t.shape != w[0].shape or t.dtype != w[0].dtype:
            raise ValueError(f"{fn}: the experts' weights must be contiguous, alike, and live on the rows' GPU")
    return (ctypes.c_void_p * len(w))(*[t.data_ptr() for t in w]), len(w), tuple(w[0].shape), w[0].dtype


def _mxfp4_rows(fn, x, x_scale):
    """(act dtype, K) of rows given in bf16 [R, K], or as MXFP4 codes [R, K/2] with scales [R, K/32]."""
    if x.dim() != 2:
        raise ValueError(f"{fn}: rows must be 2-D")
    if x.dtype == torch.bfloat16:
        return MOE_BF16, x.shape[1]
    if x.dtype != torch.uint8 or x_scale is None or x_scale.dtype != torch.uint8 \
            or x_scale.shape != (x.shape[0], x.shape[1] // 16):
        raise ValueError(f"{fn}: rows must be bfloat16 [R, K], or MXFP4 codes uint8 [R, K/2] with scales uint8 [R, K/32]")
    return MOE_MXFP4, 2 * x.shape[1]


def _mxfp4_weight(fn, w, scale, N, K, dev, masters=False):
    """Tables of E weights [N, K] given as MXFP4 codes [E, N, K/2] with scales [E, N, K/32] (or, where
    masters are taken, bf16 [E, N, K]) -> (codes table, scale table, storage dtype, E, N)."""
    t, E, shape, dtype = _weight_table(fn, w, dev)
    if masters and dtype == torch.bfloat16:
        if len(shape) != 2 or shape[1] != K or (N is not None and shape[0] != N):
            raise ValueError(f"{fn}: weight shapes do not fit the rows")
        return t, None, MOE_BF16, E, shape[0]
    if scale is None:
        raise ValueError(f"{fn}: MXFP4 weights need their scales")
    ts, Es, sshape, sdtype = _weight_table(fn, scale, dev)
    if dtype != torch.uint8 or sdtype != torch.uint8 or Es != E or len(shape) != 2 or shape[1] * 2 != K \
            or sshape != (shape[0], K // 32) or (N is not None and shape[0] != N):
        raise ValueError(f"{fn}: MXFP4 weights must be uint8 codes [N, K/2] with uint8 scales [N, K/32] per expert")
    return t, ts, MOE_MXFP4, E, shape[0]


def _check_offsets(fn, offsets, E):
    if offsets.dtype != torch.int32 or offsets.numel() != E + 1:
        raise ValueError(f"{fn}: offsets must be int32 [E + 1]")


def moe_grouped_linear_mxfp4(x: torch.Tensor, w, w_scale, offsets: torch.Tensor, x_scale: torch.Tensor | None = None,
                             out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """GroupedLinear with MXFP4 weights: y[r] = x[r] W_e^T for the rows of expert e, y [R, N] bf16.

    x: bf16 [R, K] (quantised in the call) or MXFP4 codes uint8 [R, K/2] with x_scale [R, K/32];
    w [E, N, K/2] codes with w_scale [E, N, K/32], or a list of per-expert tensors each."""
    fn = "moe_grouped_linear_mxfp4"
    _need(fn, x, offsets, x_scale, out, workspace)
    act, K = _mxfp4_rows(fn, x, x_scale)
    R = x.shape[0]
    t, ts, _, E, N = _mxfp4_weight(fn, w, w_scale, None, K, x.get_device())
    _check_offsets(fn, offsets, E)
    if out is None:
        out = torch.empty((R, N), dtype=torch.bfloat16, device=x.device)
    elif out.dtype != torch.bfloat16 or out.shape != (R, N):
        raise ValueError(f"{fn}: out must be bfloat16 [R, N]")
    need = _size(_lib.MOE_OP_LINEAR_MXFP4, (E, K, N, MOE_MXFP4, act, MOE_MXFP4, 0), R)
    if workspace is None or workspace.numel() < need:
        workspace = _workspace(need, x.device) if need else None
    _launch(fn, x, E, R, K, N, act, _a(x), _a(x_scale), t, ts, _a(offsets), _a(out), _a(workspace), need)
    return out


def _mlp_fwd_mxfp4(x, w_gate_up, w_down, offsets, prob, save_for_bwd, x_scale, w1_scale, w2_scale, out, workspace):
    fn = "moe_grouped_mlp_fwd"
    _need(fn, x, offsets, prob, x_scale, out, workspace)
    act, H = _mxfp4_rows(fn, x, x_scale)
    dev, R = x.get_device(), x.shape[0]
    t1, s1, wt, E, twoI = _mxfp4_weight(fn, w_gate_up, w1_scale, None, H, dev, masters=True)
    I = twoI // 2
    t2, s2, wt2, E2, _ = _mxfp4_weight(fn, w_down, w2_scale, H, I, dev, masters=True)
    _check_offsets(fn, offsets, E)
    if wt2 != wt or E2 != E or twoI % 2 or prob.dtype != torch.float32 or prob.numel() != R:
        raise ValueError(f"{fn}: weights must share E and storage, prob_perm must be float32 [R]")
    if out is None:
        out = torch.empty((R, H), dtype=torch.bfloat16, device=x.device)
    elif out.dtype != torch.bfloat16 or out.shape != (R, H):
        raise ValueError(f"{fn}: out must be bfloat16 [R, H]")
    desc = (E, H, I, MOE_MXFP4, act, wt, int(save_for_bwd))
    need = _size(_lib.MOE_OP_MLP_FWD, desc, R)
    if workspace is None or workspace.numel() < need:
        workspace = _workspace(need, x.device) if need else None
    _launch("moe_grouped_mlp_fwd_tables", x, ctypes.byref(MlpDesc(*desc)), R, _a(x), _a(x_scale), t1, t2, s1, s2, _a(offsets),
            _a(prob), _a(out), None, None, _a(workspace), need)
    return out


_COMPUTE = {"f32": MOE_F32, "bf16": MOE_BF16, "mxfp8": MOE_MXFP8, "fp8": MOE_FP8, "mxfp4": MOE_MXFP4}


def moe_grouped_mlp_fwd(x_perm: torch.Tensor, w_gate_up, w_down, offsets: torch.Tensor, prob_perm: torch.Tensor,
                        compute: str = "bf16", save_for_bwd: bool = False, x_perm_scale=None,
                        w_gate_up_scale=None, w_down_scale=None, out: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None):
    """Grouped MLP forward on permuted rows. Returns y_perm, or (y_perm, z, h) with save_for_bwd.

    compute: "f32", "bf16", "mxfp8", "fp8" (per-tensor scales) or "mxfp4" (forward only).
    For mxfp8, fp8 and mxfp4, x_perm may be bf16 (quantised in the call) or uint8 codes with
    x_perm_scale; weights may be bf16 master weights (quantised in the call) or uint8 codes
    with per-expert scale tensors (fp8: one float32 scale tensor per expert weight; mxfp4:
    codes [E, N, K/2] and scales [E, N, K/32] of mxfp4_quantize).
    """
    if compute == "mxfp4":
        return _mlp_fwd_mxfp4(x_perm, w_gate_up, w_down, offsets, prob_perm, save_for_bwd, x_perm_scale,
                              w_gate_up_scale, w_down_scale, out, workspace)
    w1 = _experts(w_gate_up)
    w2 = _experts(w_down)
    E = len(w1)
    twoI, H = w1[0].shape
    I = twoI // 2
    R = x_perm.shape[0]
    dev = x_perm.device
    _need_cuda(x_perm, offsets, prob_perm, x_perm_scale, *w1, *w2)
    c = _COMPUTE[compute]
    act = c if x_perm.dtype == torch.uint8 else _DT[x_perm.dtype]
    wt = c if w1[0].dtype == torch.uint8 else _DT[w1[0].dtype]
    desc = MlpDesc(E, H, I, c, act, wt, int(save_for_bwd))
    out_dtype = torch.float32 if c == MOE_F32 else torch.bfloat16
    y = out if out is not None else torch.empty((R, H), dtype=out_dtype, device=dev)
    z = torch.empty((R, 2 * I), dtype=out_dtype, device=dev) if save_for_bwd else None
    h = torch.empty((R, I), dtype=out_dtype, device=dev) if save_for_bwd else None
    need = workspace_size(_lib.MOE_OP_MLP_FWD, desc, R)
    ws = workspace if workspace is not None and workspace.numel() >= need else _workspace(need, dev)
    t1, k1 = ptr_table([t.data_ptr() for t in w1])
    t2, k2 = ptr_table([t.data_ptr() for t in w2])
    s1 = s2 = None
    keep = []
    if w_gate_up_scale is not None:
        s1, a = ptr_table([t.data_ptr() for t in _experts(w_gate_up_scale)])
        keep.append(a)
        s2, a = ptr_table([t.data_ptr() for t in _experts(w_down_scale)])
        keep.append(a)
    check("moe_grouped_mlp_fwd", lib().moe_grouped_mlp_fwd(
        ctypes.byref(desc), R, _p(x_perm), _p(x_perm_scale), t1, t2, s1, s2, _p(offsets), _p(prob_perm), _p(y),
        _p(z), _p(h), _p(ws), ws.numel(), _stream(dev)))
    del k1, k2, keep
    return (y, z, h) if save_for_bwd else y


def moe_grouped_mlp_bwd(dy_perm, x_perm, z, h, prob_perm, w_gate_up, w_down, offsets, compute: str = "bf16",
                        dw_gate_up=None, dw_down=None, workspace: torch.Tensor | None = None):
    """Grouped MLP backward. Returns (dx_perm, dw_gate_up [E, 2I, H], dw_down [E, H, I], dprob_perm [R]).

    With compute="mxfp8" the weights may be bf16 or packed by mxfp8_pack_weight_bwd (uint8); with
    compute="fp8", bf16 or packed by fp8_tensor_pack_weight_bwd (uint8)."""
    w1 = _experts(w_gate_up)
    w2 = _experts(w_down)
    E = len(w1)
    H = x_perm.shape[1]
    I = z.shape[1] // 2
    twoI = 2 * I
    R = x_perm.shape[0]
    dev = x_perm.device
    _need_cuda(dy_perm, x_perm, z, h, prob_perm, offsets, *w1, *w2)
    c = _COMPUTE[compute]
    dt = torch.float32 if c == MOE_F32 else torch.bfloat16
    wt = c if w1[0].dtype == torch.uint8 else _DT[w1[0].dtype]    # uint8: the compute dtype's packs
    desc = MlpDesc(E, H, I, c, _DT[x_perm.dtype], wt, 1)
    dx = torch.empty((R, H), dtype=dt, device=dev)
    dw1 = dw_gate_up if dw_gate_up is not None else torch.empty((E, twoI, H), dtype=dt, device=dev)
    dw2 = dw_down if dw_down is not None else torch.empty((E, H, I), dtype=dt, device=dev)
    dprob = torch.empty(R, dtype=torch.float32, device=dev)
    need = workspace_size(_lib.MOE_OP_MLP_BWD, desc, R)
    ws = workspace if workspace is not None and workspace.numel() >= need else _workspace(need, dev)
    t1, k1 = ptr_table([t.data_ptr() for t in w1])
    t2, k2 = ptr_table([t.data_ptr() for t in w2])
    d1, k3 = ptr_table([t.data_ptr() for t in _experts(dw1)])
    d2, k4 = ptr_table([t.data_ptr() for t in _experts(dw2)])
    check("moe_grouped_mlp_bwd", lib().moe_grouped_mlp_bwd(
        ctypes.byref(desc), R, _p(dy_perm), _p(x_perm), _p(z), _p(h), _p(prob_perm), t1, t2, _p(offsets), _p(dx),
        d1, d2, _p(dprob), _p(ws), ws.numel(), _stream(dev)))
    del k1, k2, k3, k4
    return dx, dw1, dw2, dprob


def _bf16_weights(fn, w_gate_up, w_down, H, dev):
    """Tables of the experts' bf16 weights [2I, H] and [H, I] -> (table, table, E, I)."""
    t1, E, shape1, dtype1 = _weight_table(fn, w_gate_up, dev)
    t2, E2, shape2, dtype2 = _weight_table(fn, w_down, dev)
    if dtype1 != torch.bfloat16 or dtype2 != torch.bfloat16 or E2 != E or len(shape2) != 2 \
            or shape1 != (2 * shape2[1], H) or shape2[0] != H:
        raise ValueError(f"{fn}: weights must be bfloat16, [2I, H] and [H, I] for each of E experts")
    return t1, t2, E, shape2[1]


def _check_prob(fn, prob, R):
    if prob.dtype != torch.float32 or prob.numel() != R:
        raise ValueError(f"{fn}: prob_perm must be float32 [R]")


def _bf16_out(fn, t, shape, dev):
    if t is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=dev)
    if t.dtype != torch.bfloat16 or t.shape != shape:
        raise ValueError(f"{fn}: an output must be bfloat16 {list(shape)}")
    return t


def moe_grouped_mlp_fwd_ckpt8(x_perm: torch.Tensor, w_gate_up, w_down, offsets: torch.Tensor, prob_perm: torch.Tensor,
                              out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """moe_grouped_mlp_fwd in bf16 that keeps its gate_up output in MXFP8 for moe_grouped_mlp_bwd_ckpt8, and
    nothing else. Returns (y_perm [R, H], z_codes uint8 [R, 2I], z_scales uint8 [R, 2I / 32]).

    y_perm is that of moe_grouped_mlp_fwd up to the order of its sums; rows past the last expert's are not written."""
    fn = "moe_grouped_mlp_fwd_ckpt8"
    _need(fn, x_perm, offsets, prob_perm, out, workspace)
    if x_perm.dtype != torch.bfloat16 or x_perm.dim() != 2:
        raise ValueError(f"{fn}: x_perm must be bfloat16 [R, H]")
    R, H = x_perm.shape
    dev = x_perm.device
    t1, t2, E, I = _bf16_weights(fn, w_gate_up, w_down, H, x_perm.get_device())
    _check_offsets(fn, offsets, E)
    _check_prob(fn, prob_perm, R)
    out = _bf16_out(fn, out, (R, H), dev)
    zc = torch.empty((R, 2 * I), dtype=torch.uint8, device=dev)
    zs = torch.empty((R, 2 * I // 32), dtype=torch.uint8, device=dev)
    desc = (E, H, I, MOE_BF16, MOE_BF16, MOE_BF16, 0)
    need = _size(_lib.MOE_OP_MLP_FWD, desc, R)
    if workspace is None or workspace.numel() < need:
        workspace = _workspace(need, dev)
    _launch(fn, x_perm, ctypes.byref(MlpDesc(*desc)), R, _a(x_perm), t1, t2, _a(offsets), _a(prob_perm), _a(out), _a(zc),
            _a(zs), _a(workspace), need)
    return out, zc, zs


def moe_grouped_mlp_bwd_ckpt8(dy_perm: torch.Tensor, x: torch.Tensor, z_codes: torch.Tensor, z_scales: torch.Tensor,
                              prob_perm: torch.Tensor, w_gate_up, w_down, offsets: torch.Tensor,
                              x_scale: torch.Tensor | None = None, src_token: torch.Tensor | None = None,
                              dx_perm: torch.Tensor | None = None, dw_gate_up: torch.Tensor | None = None,
                              dw_down: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Backward of moe_grouped_mlp_fwd_ckpt8 from what was kept. Returns (dx_perm [R, H], dw_gate_up [E, 2I, H],
    dw_down [E, H, I], dprob_perm [R] float32).

    x: the block's rows as kept: MXFP8 codes uint8 [T, H] with x_scale uint8 [T, H / 32], one row a token, and
    src_token int32 [R] (moe_permute's), or codes [R, H] in expert order without src_token; or x_perm bf16 [R, H].
    h is computed again from z. Rows of dx_perm and dprob_perm past the last expert's are not written."""
    fn = "moe_grouped_mlp_bwd_ckpt8"
    _need(fn, dy_perm, x, x_scale, src_token, z_codes, z_scales, prob_perm, offsets, dx_perm, dw_gate_up, dw_down, workspace)
    if dy_perm.dtype != torch.bfloat16 or dy_perm.dim() != 2:
        raise ValueError(f"{fn}: dy_perm must be bfloat16 [R, H]")
    R, H = dy_perm.shape
    dev = dy_perm.device
    t1, t2, E, I = _bf16_weights(fn, w_gate_up, w_down, H, dy_perm.get_device())
    _check_offsets(fn, offsets, E)
    _check_prob(fn, prob_perm, R)
    if z_codes.dtype != torch.uint8 or z_codes.shape != (R, 2 * I) or z_scales.dtype != torch.uint8 \
            or z_scales.shape != (R, 2 * I // 32):
        raise ValueError(f"{fn}: z_codes must be uint8 [R, 2I] and z_scales uint8 [R, 2I/32]")
    if x.dim() != 2 or x.shape[1] != H:
        raise ValueError(f"{fn}: x must have H columns")
    T = x.shape[0]
    if x.dtype == torch.uint8:
        act = MOE_MXFP8
        if x_scale is None or x_scale.dtype != torch.uint8 or x_scale.shape != (T, H // 32):
            raise ValueError(f"{fn}: x in 8 bits needs x_scale uint8 [T, H/32]")
        if (src_token is None and T != R) or (src_token is not None and (src_token.dtype != torch.int32
                                                                         or src_token.numel() != R)):
            raise ValueError(f"{fn}: x in 8 bits needs src_token int32 [R], or a row for every routed row")
    else:
        act = MOE_BF16
        if x.dtype != torch.bfloat16 or T != R or x_scale is not None or src_token is not None:
            raise ValueError(f"{fn}: x must be MXFP8 codes with x_scale, or bfloat16 [R, H] without x_scale and src_token")
    dx = _bf16_out(fn, dx_perm, (R, H), dev)
    dw1 = _bf16_out(fn, dw_gate_up, (E, 2 * I, H), dev)
    dw2 = _bf16_out(fn, dw_down, (E, H, I), dev)
    dprob = torch.empty(R, dtype=torch.float32, device=dev)
    d1, d2 = _weight_table(fn, dw1, dy_perm.get_device())[0], _weight_table(fn, dw2, dy_perm.get_device())[0]
    desc = (E, H, I, MOE_BF16, act, MOE_BF16, 0)
    need = _size(_lib.MOE_OP_MLP_BWD_CKPT8, desc, R)
    if workspace is None or workspace.numel() < need:
        workspace = _workspace(need, dev)
    _launch(fn, dy_perm, ctypes.byref(MlpDesc(*desc)), R, _a(dy_perm), _a(x), _a(x_scale), T, _a(src_token), _a(z_codes),
            _a(z_scales), _a(prob_perm), t1, t2, _a(offsets), _a(dx), d1, d2, _a(dprob), _a(workspace), need)
    return dx, dw1, dw2, dprob


def gemm_workspace(device) -> torch.Tensor:
    """A workspace for moe_grouped_linear / moe_grouped_gate_up_swiglu (split-K tail area)."""
    return _workspace(workspace_size(_lib.MOE_OP_GROUPED_GEMM, None, 0), device)


def moe_grouped_linear(x: torch.Tensor, w, offsets: torch.Tensor, out: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None):
    """GroupedLinear: y[r] = x[r] W_e^T for the rows of expert e. x [R, K], W_e [N, K] -> y [R, N].

    workspace: optional (see gemm_workspace); without it no tile is split along K.
    """
    ws = _experts(w)
    E = len(ws)
    N, K = ws[0].shape
    R = x.shape[0]
    _need_cuda(x, offsets, *ws)
    y = out if out is not None else torch.empty((R, N), dtype=x.dtype, device=x.device)
    t, keep = ptr_table([t.data_ptr() for t in ws])
    nws = workspace.numel() if workspace is not None else 0
    check("moe_grouped_linear", lib().moe_grouped_linear(E, R, K, N, _DT[x.dtype], _p(x), t, _p(offsets), _p(y),
                                                         _p(workspace), nws, _stream(x.device)))
    del keep
    return y


def moe_grouped_gate_up_swiglu(x: torch.Tensor, w_gate_up, offsets: torch.Tensor, prob: torch.Tensor,
                               save_z: bool = False, x_scale=None, w_scale=None, out: torch.Tensor | None = None,
                               out_scale: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """GroupedLinear(gate_up) fused with ScaledSwiGLU: h = silu(x W_e[:I]^T) * (x W_e[I:]^T) * prob.

    bf16/f32: returns h [R, I] (and z [R, 2I] with save_z). MXFP8 (x given as uint8 codes
    with x_scale, weights as codes with w_scale): returns (h codes [R, I], h scales [R, I/32]).
    """
    ws = _experts(w_gate_up)
    E = len(ws)
    twoI, H = ws[0].shape
    I = twoI // 2
    R = x.shape[0]
    dev = x.device
    _need_cuda(x, offsets, prob, x_scale, *ws)
    dt = _DT[x.dtype]
    t, keep = ptr_table([t.data_ptr() for t in ws])
    st = None
    if dt == MOE_MXFP8:
        st, keep2 = ptr_table([t.data_ptr() for t in _experts(w_scale)])
        h = out if out is not None else torch.empty((R, I), dtype=torch.uint8, device=dev)
        hs = out_scale if out_scale is not None else torch.empty((R, I // 32), dtype=torch.uint8, device=dev)
        z = None
    else:
        h = out if out is not None else torch.empty((R, I), dtype=x.dtype, device=dev)
        hs = None
        z = torch.empty((R, twoI), dtype=x.dtype, device=dev) if save_z else None
    check("moe_grouped_gate_up_swiglu", lib().moe_grouped_gate_up_swiglu(
        E, R, H, I, dt, _p(x), _p(x_scale), t, st, _p(offsets), _p(prob), _p(h), _p(hs), _p(z), _p(workspace),
        workspace.numel() if workspace is not None else 0, _stream(dev)))
    del keep
    if dt == MOE_MXFP8:
        return h, hs
    return (h, z) if save_z else h
