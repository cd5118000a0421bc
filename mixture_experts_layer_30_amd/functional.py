"""Buffer allocation around the C ABI, in the shape of the functional API the
MoK project card describes (get_workspace -> build_schedule -> forward ->
backward). torch provides the device memory; every computation happens in
libmok's kernels.
"""
from __future__ import annotations

import dataclasses
from typing import NamedTuple

import torch

from . import (ACT_SILU, MOK_BF16, backward, buffer_sizes, build_schedule, ffn_backward, ffn_buffer_sizes,
               ffn_forward, forward, forward_fused, make_config, make_ffn_problem, make_mx_problem, make_problem,
               make_norm_problem, mx_matmul, mx_matmul_workspace, mxfp8_quantize, mxfp8_quantize_transposed,
               norm_backward, norm_forward, norm_workspace, router_forward_logits, router_logits_backward,
               router_workspace, schedule_layout)
from . import mxfp4_dequantize as _mxfp4_dequantize
from . import mxfp4_quantize as _mxfp4_quantize
from . import mxfp8_dequantize as _mxfp8_dequantize
# the calls below that allocate their outputs leave out the checks of those
from . import (_device_of, _norm_backward, _norm_forward, _router_logits_backward, _router_losses,
               _router_losses_backward)


@dataclasses.dataclass
class Workspace:
    problem: object
    config: object
    workspace: torch.Tensor
    schedule: torch.Tensor
    fwd_ctx: torch.Tensor | None


def get_workspace(T, H, I, E, topk, dtype=MOK_BF16, device="cuda", training=True, **cfg):
    """Allocate the workspace, schedule and fwd_ctx buffers for one layer shape."""
    problem = make_problem(T, H, I, E, topk, dtype)
    config = make_config(**cfg)
    ws, sb, cb = buffer_sizes(problem, config)
    mk = lambda n: torch.empty(max(int(n), 16), dtype=torch.uint8, device=device)  # noqa: E731
    return Workspace(problem, config, mk(ws), mk(sb), mk(cb) if (training and cb) else None)


def run_schedule(w: Workspace, topk_ids):
    build_schedule(w.problem, topk_ids, w.schedule, w.config)


def run_forward(w: Workspace, x, topk_w, weights, y=None):
    if y is None:
        y = torch.empty_like(x)
    forward(w.problem, w.schedule, x, topk_w, weights, y, w.workspace, w.fwd_ctx, w.config)
    return y


def run_forward_fused(w: Workspace, topk_ids, x, topk_w, weights, y=None):
    """Schedule + forward in one persistent launch (mok_forward_fused)."""
    if y is None:
        y = torch.empty_like(x)
    forward_fused(w.problem, topk_ids, w.schedule, x, topk_w, weights, y, w.workspace, w.fwd_ctx, w.config)
    return y


def run_backward(w: Workspace, x, topk_w, weights, dy):
    wg, wu, wd = weights[:3]
    dx = torch.empty_like(x)
    dwg, dwu, dwd = torch.empty_like(wg), torch.empty_like(wu), torch.empty_like(wd)
    dtw = torch.empty_like(topk_w)
    backward(w.problem, w.schedule, w.fwd_ctx, x, topk_w, weights, dy, dx, dwg, dwu, dwd, dtw,
             w.workspace, w.config)
    return dx, dwg, dwu, dwd, dtw


def quantize_weights_backward(wg, wu, wd):
    """The MXFP8 weight copies the MXFP8 backward needs, quantized along the
    weights' other axis by the library's transposing quantizer: Wd^T
    [E][I][H] blocked along H, and [Wg; Wu]^T [E][H][2I] blocked along 2I
    (Wg into columns [0, I), Wu into [I, 2I)).
    Returns (w_down_t, w_gu_t, s_down_t, s_gu_t)."""
    E, I, H = wg.shape
    dev = wg.device
    qd = torch.empty((E, I, H), dtype=torch.uint8, device=dev)
    sd = torch.empty((E, I, H // 32), dtype=torch.uint8, device=dev)
    qgu = torch.empty((E, H, 2 * I), dtype=torch.uint8, device=dev)
    sgu = torch.empty((E, H, 2 * I // 32), dtype=torch.uint8, device=dev)
    mxfp8_quantize_transposed(wd, qd, sd)
    mxfp8_quantize_transposed(wg, qgu, sgu, col0=0)
    mxfp8_quantize_transposed(wu, qgu, sgu, col0=I)
    return qd, qgu, sd, sgu


def quantize_weights(wg, wu, wd):
    """MXFP8 copies of the expert weights along their contraction axes."""
    out = []
    for m in (wg, wu, wd):
        q = torch.empty(m.shape, dtype=torch.uint8, device=m.device)
        s = torch.empty(m.shape[:-1] + (m.shape[-1] // 32,), dtype=torch.uint8, device=m.device)
        mxfp8_quantize(m.reshape(-1, m.shape[-1]), q, s)
        out.append((q, s))
    (qg, sg), (qu, su), (qd, sd) = out
    return qg, qu, qd, sg, su, sd


def read_schedule(w: Workspace):
    """Copy the schedule arrays to the host (for inspection and tests)."""
    L = schedule_layout(w.problem, w.config)
    s = w.schedule.cpu()
    E, R = w.problem.E, w.problem.T * w.problem.topk

    def arr(off, n):
        return s[off:off + 4 * n].view(torch.int32).numpy().copy()

    nf = int(arr(L.n_fwd_tiles, 1)[0])
    nb = int(arr(L.n_bwd_tiles, 1)[0])
    return {
        "status": int(arr(L.status, 1)[0]),
        "counts": arr(L.counts, E),
        "offsets": arr(L.offsets, E + 1),
        "perm": arr(L.perm, R),
        "dest": arr(L.dest, R),
        "fwd_tiles": arr(L.fwd_tiles, 4 * nf).reshape(nf, 4),
        "mb_tile_start": arr(L.mb_tile_start, L.n_minibatches + 1),
        "bwd_tiles": arr(L.bwd_tiles, 4 * nb).reshape(nb, 4),
        "expert_order": arr(L.expert_order, E),
        "M": L.minibatch_rows, "n_slots": L.ring_slots, "n_mb": L.n_minibatches,
        "fwd_tile_rows": L.fwd_tile_rows, "bwd_tile_rows": L.bwd_tile_rows,
    }


# ---------------------------------------------------------------- MXFP4 and the dense block
def mxfp4_quantize(src):
    """(codes [..., K/2], scales [..., K/32]) of the bf16 rows of src [..., K]."""
    q = torch.empty((*src.shape[:-1], src.shape[-1] // 2), dtype=torch.uint8, device=src.device)
    s = torch.empty((*src.shape[:-1], src.shape[-1] // 32), dtype=torch.uint8, device=src.device)
    _mxfp4_quantize(src, q, s)
    return q, s


def mxfp4_dequantize(q, scales):
    """The bf16 values [..., K] of MXFP4 codes and scales."""
    out = torch.empty((*q.shape[:-1], 2 * q.shape[-1]), dtype=torch.bfloat16, device=q.device)
    _mxfp4_dequantize(q, scales, out)
    return out


@dataclasses.dataclass
class MxWorkspace:
    problem: object
    workspace: torch.Tensor | None


def get_mx_matmul_workspace(M, N, K, a_dtype, device="cuda"):
    """The problem and scratch of one product shape."""
    problem = make_mx_problem(M, N, K, a_dtype)
    n = mx_matmul_workspace(problem)
    return MxWorkspace(problem, torch.empty(n, dtype=torch.uint8, device=device) if n else None)


def run_mx_matmul(w: MxWorkspace, a, a_scales, b, b_scales, out=None):
    """out [M][N] bf16 = A . B^T, B in MXFP4, A in the workspace's a_dtype."""
    if out is None:
        out = torch.empty((w.problem.M, w.problem.N), dtype=torch.bfloat16, device=a.device)
    mx_matmul(w.problem, a, a_scales, b, b_scales, out, w.workspace)
    return out


@dataclasses.dataclass
class FfnWorkspace:
    problem: object
    workspace: torch.Tensor
    ctx: torch.Tensor | None     # [T][2I] bf16: the pre-activations a | b of the last forward


def get_ffn_workspace(T, H, I, dtype=MOK_BF16, activation=ACT_SILU, device="cuda", training=True):
    """Allocate the workspace and (training) the saved context of one dense block; without training, the workspace
    of forwards alone, and run_ffn_backward refuses it."""
    problem = make_ffn_problem(T, H, I, dtype, activation, forward_only=not training)
    ws, cb = ffn_buffer_sizes(problem)
    ctx = torch.empty((T, 2 * I), dtype=torch.bfloat16, device=device) if training and dtype == MOK_BF16 else None
    return FfnWorkspace(problem, torch.empty(max(ws, 16), dtype=torch.uint8, device=device), ctx)


def run_ffn_forward(w: FfnWorkspace, x, weights, residual=None, y=None):
    """y = block(x) (+ residual, which may be the y passed in); saves the context if the workspace holds one."""
    if y is None:
        y = torch.empty((x.shape[0], x.shape[1]), dtype=x.dtype, device=x.device)
    ffn_forward(w.problem, x, weights, y, w.workspace, residual=residual, ctx=w.ctx)
    return y


def run_ffn_backward(w: FfnWorkspace, x, weights, dy):
    """(dx, dw_gate, dw_up, dw_down) from the context of the last forward."""
    wg, wu, wd = weights[:3]
    dx = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=x.device)
    dwg, dwu, dwd = torch.empty_like(wg), torch.empty_like(wu), torch.empty_like(wd)
    ffn_backward(w.problem, w.ctx, x, weights, dy, dx, dwg, dwu, dwd, w.workspace)
    return dx, dwg, dwu, dwd


def quantize_ffn_weights_mxfp4(wg, wu, wd):
    """The six tensors a dense block with MXFP4 weights takes (codes, then scales)."""
    (qg, sg), (qu, su), (qd, sd) = (mxfp4_quantize(m) for m in (wg, wu, wd))
    return qg, qu, qd, sg, su, sd


# ---------------------------------------------------------------- the norm before the layer
def mxfp8_dequantize(q, scales):
    """The bf16 values [..., K] of MXFP8 codes and scales."""
    out = torch.empty_like(q, dtype=torch.bfloat16, memory_format=torch.contiguous_format)
    _mxfp8_dequantize(q, scales, out)
    return out


@dataclasses.dataclass
class NormWorkspace:
    problem: object
    workspace: torch.Tensor | None
    training: bool


class NormOutput(NamedTuple):
    y: torch.Tensor | None       # [T][H] bf16
    sum: torch.Tensor | None     # [T][H] bf16: the residual stream (x itself without a residual; None: y lies over it)
    rstd: torch.Tensor | None    # [T] fp32, in training
    q: torch.Tensor | None       # [T][H] MXFP8 codes of y, and
    scales: torch.Tensor | None  # [T][H/32] their scales


def get_norm_workspace(T, H, eps=1e-6, weight_dtype=torch.bfloat16, device="cuda", training=True):
    """The problem and (training) the backward's scratch of one norm."""
    if weight_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"weight_dtype: {weight_dtype}, wanted torch.bfloat16 or torch.float32")
    problem = make_norm_problem(T, H, eps, weight_dtype == torch.float32)
    n = norm_workspace(problem) if training else 0
    return NormWorkspace(problem, torch.empty(n, dtype=torch.uint8, device=device) if n else None, training)


def run_norm_forward(w: NormWorkspace, x, weight, residual=None, out="bf16", y=None, sum_out=None):
    """The norm of x, or of the stream x + residual, which is returned too (sum_out=residual updates it in place).
    out: "bf16" (y), "mxfp8" (q and scales, as run_mx_matmul takes them) or "both". weight None: ones. y=x without a
    residual overwrites the stream, which a backward needs: sum is None then."""
    if out not in ("bf16", "mxfp8", "both"):
        raise ValueError(f"out: {out!r}, wanted 'bf16', 'mxfp8' or 'both'")
    given = y is not None or sum_out is not None
    dense = x.is_contiguous()                    # (the cheapest way to an output of x's shape)
    q = scales = rstd = None
    if out == "mxfp8":
        if y is not None:
            raise ValueError("y: not written with out='mxfp8'")
    elif y is None:
        y = torch.empty_like(x) if dense else x.new_empty(x.shape)
    if out != "bf16":
        q = torch.empty_like(x, dtype=torch.uint8) if dense else x.new_empty(x.shape, dtype=torch.uint8)
        scales = x.new_empty((w.problem.T, w.problem.H // 32), dtype=torch.uint8)
    if residual is not None and sum_out is None:
        sum_out = _rows_like(residual)
    if w.training:
        rstd = x.new_empty(w.problem.T, dtype=torch.float32)
    if given:
        norm_forward(w.problem, x, weight, y, residual, sum_out, rstd, q, scales)
    else:
        _norm_forward(w.problem, _device_of(x), x, weight, y, residual, sum_out, rstd, q, scales, None)
    if residual is None:
        sum_out = None if given and x.numel() and y.data_ptr() == x.data_ptr() else x
    return NormOutput(y, sum_out, rstd, q, scales)


def _rows_like(t):
    """An empty tensor of t's shape and row pitch."""
    if t.is_contiguous():
        return torch.empty_like(t)
    return torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=t.device)


def run_norm_backward(w: NormWorkspace, z, rstd, weight, dy, d_sum=None, dx=None):
    """(dx, dw) from the forward's sum (z) and rstd; d_sum, the gradient that reaches the stream from further on, is
    added to dx. dw is None without a weight."""
    if not w.training:
        raise ValueError("a norm workspace without training has no backward")
    if z is None:
        raise ValueError("z: None, the stream that the forward normed is wanted (y was written over it)")
    dw = None if weight is None else torch.empty_like(weight)
    if dx is not None:
        norm_backward(w.problem, dy, z, rstd, weight, dx, dw, w.workspace, d_sum=d_sum)
    else:
        dx = _rows_like(dy if d_sum is None else d_sum)
        _norm_backward(w.problem, _device_of(dy), dy, z, rstd, weight, dx, dw, w.workspace, d_sum, None)
    return dx, dw


# ---------------------------------------------------------------- the router in training, with its losses
@dataclasses.dataclass
class RouterWorkspace:
    problem: object
    workspace: torch.Tensor | None


class RouterLosses(NamedTuple):
    losses: torch.Tensor         # [2] fp32: balance loss, z loss
    counts: torch.Tensor         # [E] int32: picks of each expert
    prob_sum: torch.Tensor       # [E] fp32: summed probabilities
    n_tokens: torch.Tensor       # [1] int32: tokens that the mask kept


def get_router_workspace(T, H, E, topk, device="cuda"):
    """The problem and scratch of one router's losses and backward."""
    problem = make_problem(T, H, 128, E, topk)
    n = router_workspace(problem)
    return RouterWorkspace(problem, torch.empty(n, dtype=torch.uint8, device=device) if n else None)


def run_router_forward(w: RouterWorkspace, x, w_router, bias=None):
    """(topk_ids, topk_w, logits) of the tokens x."""
    p = w.problem
    ids = torch.empty((p.T, p.topk), dtype=torch.int32, device=x.device)
    tw = torch.empty((p.T, p.topk), dtype=torch.float32, device=x.device)
    logits = torch.empty((p.T, p.E), dtype=torch.float32, device=x.device)
    router_forward_logits(p, x, w_router, bias, ids, tw, logits)
    return ids, tw, logits


def run_router_losses(w: RouterWorkspace, logits, topk_ids, mask=None):
    """The balance and z losses of the tokens that mask [T] keeps (None: all), and the sums under them."""
    E = w.problem.E
    out = RouterLosses(logits.new_empty(2), topk_ids.new_empty(E), logits.new_empty(E), topk_ids.new_empty(1))
    _router_losses(w.problem, _device_of(logits), logits, topk_ids, *out, w.workspace, mask, None)
    return out


def run_router_losses_backward(w: RouterWorkspace, logits, topk_ids, sums: RouterLosses, d_losses, topk_w=None,
                               d_topk_w=None, mask=None):
    """d_logits from the gradients of the two losses (a tensor on the device) and, with topk_w and the layer's
    d_topk_w, through the combine weights. sums: what run_router_losses returned for the same mask."""
    d_logits = torch.empty_like(logits)
    _router_losses_backward(w.problem, _device_of(logits), logits, topk_ids, sums.counts, sums.n_tokens, d_losses,
                            d_logits, topk_w, d_topk_w, mask, None)
    return d_logits


def run_router_logits_backward(w: RouterWorkspace, x, w_router, d_logits, residual=None, dx=None):
    """(dx, d_w_router); residual, the layer's own dx, is added (and may be the dx passed in)."""
    dwr = torch.empty_like(w_router)
    if dx is not None:
        router_logits_backward(w.problem, x, w_router, d_logits, dx, dwr, w.workspace, residual=residual)
    else:
        dx = torch.empty_like(x)
        _router_logits_backward(w.problem, _device_of(x), x, w_router, d_logits, dx, dwr, w.workspace, residual, None)
    return dx, dwr
