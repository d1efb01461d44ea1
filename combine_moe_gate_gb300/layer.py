"""Device buffers for one MoE layer forward, allocated with torch (plumbing only).

The layer itself runs in libmoe_gate.so (`moe_layer_forward`, or the single
calls that `run_layer_fp4` makes); this module sizes and allocates the tensors
the C ABI writes into.
"""

from contextlib import nullcontext
from dataclasses import dataclass
from typing import Optional

import torch

from . import (MOE_BF16, MOE_F32, MOE_FLAG_NORMALIZE_GATES, moe_capacity_bound,
               moe_capacity_locations, moe_capacity_workspace_size, moe_decode, moe_decode_sorted,
               moe_decode_sorted_bwd, moe_encode, moe_encode_sorted, moe_encode_sorted_bwd,
               moe_expert_ffn_fp4, moe_expert_ffn_fp4_workspace_size, moe_expert_ffn_int8,
               moe_expert_ffn_int8_workspace_size, moe_expert_ffn_sorted, moe_expert_ffn_sorted_bwd,
               moe_expert_ffn_sorted_bwd_workspace_size, moe_fp4_scale_bytes, moe_layer_forward,
               moe_layer_forward_host, moe_layer_workspace_size, moe_quantize_fp4,
               moe_quantize_rows_int8, moe_route_bwd, moe_route_topk, moe_sort_routes,
               moe_sort_workspace_size)


@dataclass
class MoELayerBuffers:
    idx: torch.Tensor      # [k, s] int32
    gates: torch.Tensor    # [k, s] fp32
    loc: torch.Tensor      # [k, s] int32
    counts: torch.Tensor   # [e] int32
    c_dev: torch.Tensor    # [1] int32
    buf: torch.Tensor      # [e, c_max, m]
    out: torch.Tensor      # [e, c_max, m]
    y: torch.Tensor        # [s, m]
    workspace: torch.Tensor
    status: torch.Tensor   # [1] int32

    @property
    def c_max(self) -> int:
        return self.buf.shape[1]


def alloc_layer(s, m, e, k, h, act, capacity_factor, dtype=torch.bfloat16, device="cuda",
                c_max: Optional[int] = None) -> MoELayerBuffers:
    """Allocate every output and scratch tensor of one layer forward.

    c_max defaults to the capacity bound, which can never overflow."""
    if c_max is None:
        c_max = moe_capacity_bound(capacity_factor, s, e, k)
    dt = MOE_BF16 if dtype == torch.bfloat16 else MOE_F32
    ws = moe_layer_workspace_size(dt, act, s, m, e, k, c_max, h)
    i32 = dict(dtype=torch.int32, device=device)
    return MoELayerBuffers(
        idx=torch.empty((k, s), **i32),
        gates=torch.empty((k, s), dtype=torch.float32, device=device),
        loc=torch.empty((k, s), **i32),
        counts=torch.empty((e,), **i32),
        c_dev=torch.empty((1,), **i32),
        buf=torch.empty((e, c_max, m), dtype=dtype, device=device),
        out=torch.empty((e, c_max, m), dtype=dtype, device=device),
        y=torch.empty((s, m), dtype=dtype, device=device),
        workspace=torch.empty((ws,), dtype=torch.uint8, device=device),
        status=torch.zeros((1,), **i32),
    )


def run_layer_host(x_host, y_host, x, wg, gate_bias, w1, b1, w3, w2, b2, act, k, capacity_factor,
                   bufs: MoELayerBuffers, normalize_gates=True, flags=0, stream=None):
    """Enqueue host-to-device copy of x_host, the whole forward layer and the
    copy of y back to y_host (one C call); the caller synchronises."""
    if normalize_gates:
        flags |= MOE_FLAG_NORMALIZE_GATES
    moe_layer_forward_host(x_host, y_host, x, wg, gate_bias, w1, b1, w3, w2, b2, act, k,
                           capacity_factor, flags, bufs.idx, bufs.gates, bufs.loc, bufs.counts,
                           bufs.c_dev, bufs.buf, bufs.out, bufs.y, bufs.workspace, bufs.status,
                           stream=stream)
    return y_host


def run_layer(x, wg, gate_bias, w1, b1, w3, w2, b2, act, k, capacity_factor, bufs: MoELayerBuffers,
              normalize_gates=True, flags=0, stream=None):
    """Enqueue the whole forward layer; returns bufs.y (no host synchronisation)."""
    if normalize_gates:
        flags |= MOE_FLAG_NORMALIZE_GATES
    moe_layer_forward(x, wg, gate_bias, w1, b1, w3, w2, b2, act, k, capacity_factor, flags,
                      bufs.idx, bufs.gates, bufs.loc, bufs.counts, bufs.c_dev, bufs.buf, bufs.out,
                      bufs.y, bufs.workspace, bufs.status, stream=stream)
    return bufs.y


# --------------------------------------------- the layer on 4-bit experts
@dataclass
class Fp4Operand:
    """Rows in a microscaled 4-bit format, as moe_quantize_fp4 lays them out."""
    q: torch.Tensor                          # [e, rows, cols / 2] uint8
    scale: torch.Tensor                      # [e, moe_fp4_scale_bytes] uint8
    global_scale: Optional[torch.Tensor]     # [e] fp32 ("nv" only)


def quantize_weights_fp4(w, fmt) -> Fp4Operand:
    """4-bit form of expert weights [e, rows, cols] (bf16 or fp32), made once.
    "nv": each expert's factor is its largest finite magnitude / (6 * 448), so
    that the largest block scale is the largest e4m3 number (an infinity or a NaN
    makes its own block NaN and has no part in the factor)."""
    e, rows, cols = w.shape
    g = None
    if fmt == "nv":
        g = w.abs().nan_to_num_(nan=0.0, posinf=0.0).amax((1, 2)).float() / (6.0 * 448.0)
        g = torch.where(g > 0, g, torch.ones_like(g))
    q = torch.empty((e, rows, cols // 2), dtype=torch.uint8, device=w.device)
    scale = torch.empty((e, moe_fp4_scale_bytes(fmt, rows, cols)), dtype=torch.uint8, device=w.device)
    status = torch.zeros((1,), dtype=torch.int32, device=w.device)
    moe_quantize_fp4(w, fmt, q, scale, status, global_scale=g)
    return Fp4Operand(q, scale, g)


@dataclass
class MoELayerFp4Buffers:
    idx: torch.Tensor      # [k, s] int32
    gates: torch.Tensor    # [k, s] fp32
    loc: torch.Tensor      # [k, s] int32
    counts: torch.Tensor   # [e] int32
    c_dev: torch.Tensor    # [1] int32
    buf: torch.Tensor      # [e, c_max, m] bf16
    buf_q: torch.Tensor    # [e, c_max, m / 2] uint8
    buf_scale: torch.Tensor  # [e, moe_fp4_scale_bytes] uint8
    out: torch.Tensor      # [e, c_max, m] bf16
    y: torch.Tensor        # [s, m] bf16
    cap_ws: torch.Tensor   # moe_capacity_locations' workspace
    ffn_ws: torch.Tensor   # moe_expert_ffn_fp4's workspace
    status: torch.Tensor   # [1] int32


def alloc_layer_fp4(s, m, e, k, h, act, fmt, capacity_factor, device="cuda",
                    c_max: Optional[int] = None) -> MoELayerFp4Buffers:
    """Every output and scratch tensor of run_layer_fp4 (c_max: as alloc_layer)."""
    if c_max is None:
        c_max = moe_capacity_bound(capacity_factor, s, e, k)
    i32 = dict(dtype=torch.int32, device=device)
    u8 = dict(dtype=torch.uint8, device=device)
    bf = dict(dtype=torch.bfloat16, device=device)
    return MoELayerFp4Buffers(
        idx=torch.empty((k, s), **i32),
        gates=torch.empty((k, s), dtype=torch.float32, device=device),
        loc=torch.empty((k, s), **i32),
        counts=torch.empty((e,), **i32),
        c_dev=torch.empty((1,), **i32),
        buf=torch.empty((e, c_max, m), **bf),
        buf_q=torch.empty((e, c_max, m // 2), **u8),
        buf_scale=torch.empty((e, moe_fp4_scale_bytes(fmt, c_max, m)), **u8),
        out=torch.empty((e, c_max, m), **bf),
        y=torch.empty((s, m), **bf),
        cap_ws=torch.empty((moe_capacity_workspace_size(s, e, k),), **u8),
        ffn_ws=torch.empty((moe_expert_ffn_fp4_workspace_size(fmt, act, e, c_max, m, h),), **u8),
        status=torch.zeros((1,), **i32),
    )


def run_layer_fp4(x, logits, bias, w1: Fp4Operand, b1, w3: Optional[Fp4Operand], w2: Fp4Operand, b2,
                  fmt, act, k, capacity_factor, bufs: MoELayerFp4Buffers, buf_global=None,
                  hid_global=None, score="softmax", groups=1, topk_groups=1, group_top=1, scale=1.0,
                  normalize_gates=True, stream=None):
    """Enqueue a whole layer with routing from `logits` [s, e] (the router's
    projection of x; moe_route_topk's options) and 4-bit experts (weights from
    quantize_weights_fp4; "nv": buf_global and hid_global [e], the calibrated
    factors of the layer's input and hidden).  Returns bufs.y, with no host
    synchronisation.  A route to a masked expert (gate 0) takes a slot like any
    other: with a capacity_factor other than 0, tokens that have no expert (padding)
    are better left out of x and logits than masked."""
    B = bufs
    e = logits.shape[1]
    w3 = w3 or Fp4Operand(None, None, None)
    moe_route_topk(logits, bias, k, B.idx, B.gates, B.status, score=score, groups=groups,
                   topk_groups=topk_groups, group_top=group_top, scale=scale,
                   flags=MOE_FLAG_NORMALIZE_GATES if normalize_gates else 0, stream=stream)
    moe_capacity_locations(B.idx, e, capacity_factor, B.buf.shape[1], B.cap_ws, B.loc, B.counts,
                           B.c_dev, B.status, stream=stream)
    moe_encode(x, B.idx, B.loc, B.counts, B.c_dev, B.buf, B.status, stream=stream)
    moe_quantize_fp4(B.buf, fmt, B.buf_q, B.buf_scale, B.status, global_scale=buf_global,
                     counts=B.counts, c_dev=B.c_dev, stream=stream)
    moe_expert_ffn_fp4(B.buf_q, B.buf_scale, buf_global, hid_global, B.counts, B.c_dev, w1.q, w1.scale,
                       w1.global_scale, b1, w3.q, w3.scale, w3.global_scale, w2.q, w2.scale,
                       w2.global_scale, b2, fmt, act, B.ffn_ws, B.out, B.status, stream=stream)
    moe_decode(B.out, B.idx, B.loc, B.gates, B.c_dev, B.y, B.status, stream=stream)
    return B.y


# ------------------------------------------- the layer on rows sorted by expert
@dataclass
class MoESortedBuffers:
    idx: torch.Tensor      # [k, s] int32 (-1: a padded token's)
    gates: torch.Tensor    # [k, s] fp32
    rows: torch.Tensor     # [k, s] int32
    offsets: torch.Tensor  # [e + 1] int32
    xs: Optional[torch.Tensor]   # [s * k, m] bf16: the tokens' rows (8-bit experts: None)
    hid: Optional[torch.Tensor]  # [s * k, h] bf16
    pre: Optional[torch.Tensor]  # [s * k, h or 2h] bf16 (training)
    xs_q: Optional[torch.Tensor]      # 8-bit experts: [s * k, m] int8
    xs_scale: Optional[torch.Tensor]  # and [s * k] fp32
    out: torch.Tensor      # [s * k, m] bf16
    y: torch.Tensor        # [s, m] bf16
    sort_ws: torch.Tensor  # moe_sort_routes' workspace
    ffn_ws: Optional[torch.Tensor]    # moe_expert_ffn_int8's
    status: torch.Tensor   # [1] int32


def alloc_layer_sorted(s, m, e, k, h, act, device="cuda", train=False, int8=False) -> MoESortedBuffers:
    """Every output and scratch tensor of run_layer_sorted (train: with what its
    gradient needs) or, int8, of run_layer_int8.  No capacity: s * k rows hold
    any routing."""
    n = s * k
    i32 = dict(dtype=torch.int32, device=device)
    f32 = dict(dtype=torch.float32, device=device)
    bf = dict(dtype=torch.bfloat16, device=device)
    u8 = dict(dtype=torch.uint8, device=device)
    return MoESortedBuffers(
        idx=torch.empty((k, s), **i32),
        gates=torch.empty((k, s), **f32),
        rows=torch.empty((k, s), **i32),
        offsets=torch.empty((e + 1,), **i32),
        xs=None if int8 else torch.empty((n, m), **bf),
        hid=None if int8 else torch.empty((n, h), **bf),
        pre=torch.empty((n, 2 * h if act == "swiglu" else h), **bf) if train else None,
        xs_q=torch.empty((n, m), dtype=torch.int8, device=device) if int8 else None,
        xs_scale=torch.empty((n,), **f32) if int8 else None,
        out=torch.empty((n, m), **bf),
        y=torch.empty((s, m), **bf),
        sort_ws=torch.empty((moe_sort_workspace_size(s, e, k),), **u8),
        ffn_ws=torch.empty((moe_expert_ffn_int8_workspace_size(act, e, n, m, h),), **u8) if int8 else None,
        status=torch.zeros((1,), **i32),
    )


def _route_sorted(B, logits, bias, k, score, groups, topk_groups, group_top, scale, normalize_gates, padding, stream):
    e = logits.shape[1]
    moe_route_topk(logits, bias, k, B.idx, B.gates, B.status, score=score, groups=groups, topk_groups=topk_groups,
                   group_top=group_top, scale=scale, flags=MOE_FLAG_NORMALIZE_GATES if normalize_gates else 0,
                   stream=stream)
    if padding is not None:
        with torch.cuda.stream(stream) if stream is not None else nullcontext():
            B.idx.masked_fill_(padding, -1)
    moe_sort_routes(B.idx, e, B.rows, B.offsets, B.sort_ws, B.status, stream=stream)


def run_layer_sorted(x, logits, bias, w1, b1, w3, w2, b2, act, k, bufs: MoESortedBuffers, score="softmax", groups=1,
                     topk_groups=1, group_top=1, scale=1.0, normalize_gates=True, padding=None, stream=None):
    """Enqueue a whole layer without a capacity (no route is dropped): routing from
    `logits` [s, e] (moe_route_topk's options), the rows sorted by expert, bf16
    experts, the weighted way back.  padding [s] bool: tokens that take no expert;
    their y is 0.  Returns bufs.y, with no host synchronisation."""
    B = bufs
    _route_sorted(B, logits, bias, k, score, groups, topk_groups, group_top, scale, normalize_gates, padding, stream)
    moe_encode_sorted(x, B.rows, B.xs, B.status, stream=stream)
    moe_expert_ffn_sorted(B.xs, B.offsets, w1, b1, w3, w2, b2, act, B.hid, B.out, B.status, pre=B.pre, stream=stream)
    moe_decode_sorted(B.out, B.rows, B.y, B.status, gates=B.gates, stream=stream)
    return B.y


@dataclass
class MoESortedGrads:
    d_out: torch.Tensor     # [s * k, m] bf16: of the experts' output rows
    d_xs: torch.Tensor      # [s * k, m] bf16: of the experts' input rows
    d_gates: torch.Tensor   # [k, s] fp32
    d_logits: torch.Tensor  # [s, e] fp32
    d_x: torch.Tensor       # [s, m] bf16 (through the experts; the router's part is d_logits' caller's)
    d_w1: torch.Tensor
    d_w3: Optional[torch.Tensor]
    d_w2: torch.Tensor
    d_b1: Optional[torch.Tensor]
    d_b2: Optional[torch.Tensor]
    ffn_ws: torch.Tensor


def alloc_grads_sorted(s, k, w1, w3, w2, act, wgrad_dtype=torch.bfloat16) -> MoESortedGrads:
    """Every output and scratch tensor of run_layer_sorted_bwd; the weights' and
    biases' gradients in wgrad_dtype (bf16 or fp32).  SwiGLU takes no biases."""
    e, h, m = w1.shape
    n, dev, swiglu = s * k, w1.device, act == "swiglu"
    bf = dict(dtype=torch.bfloat16, device=dev)
    f32 = dict(dtype=torch.float32, device=dev)
    wg = dict(dtype=wgrad_dtype, device=dev)
    return MoESortedGrads(
        d_out=torch.empty((n, m), **bf), d_xs=torch.empty((n, m), **bf), d_gates=torch.empty((k, s), **f32),
        d_logits=torch.empty((s, e), **f32), d_x=torch.empty((s, m), **bf), d_w1=torch.empty(w1.shape, **wg),
        d_w3=torch.empty(w3.shape, **wg) if swiglu else None, d_w2=torch.empty(w2.shape, **wg),
        d_b1=None if swiglu else torch.empty((e, h), **wg), d_b2=None if swiglu else torch.empty((e, m), **wg),
        ffn_ws=torch.empty((moe_expert_ffn_sorted_bwd_workspace_size(act, e, n, m, h),), dtype=torch.uint8, device=dev))


def run_layer_sorted_bwd(dy, logits, w1, w3, w2, act, bufs: MoESortedBuffers, grads: MoESortedGrads, score="softmax",
                         scale=1.0, normalize_gates=True, padding=None, stream=None):
    """Enqueue the gradient of run_layer_sorted (buffers of alloc_layer_sorted with
    train=True as it left them; score, scale, normalize_gates and padding as given
    to it) for dy [s, m]: fills and returns grads."""
    B, G = bufs, grads
    moe_decode_sorted_bwd(dy, B.out, B.rows, B.gates, G.d_out, G.d_gates, B.status, stream=stream)
    moe_expert_ffn_sorted_bwd(B.xs, B.hid, B.pre, B.offsets, w1, w3, w2, act, G.d_out, G.ffn_ws, G.d_xs, G.d_w1, G.d_w3,
                              G.d_w2, G.d_b1, G.d_b2, B.status, stream=stream)
    moe_encode_sorted_bwd(G.d_xs, B.rows, G.d_x, B.status, stream=stream)
    idx = B.idx
    on = torch.cuda.stream(stream) if stream is not None else nullcontext()
    if padding is not None:   # any k different experts: these tokens' gradient is set to 0 below
        with on:
            first = torch.arange(idx.shape[0], dtype=torch.int32, device=idx.device)[:, None]
            idx = torch.where(padding, first, idx)
    moe_route_bwd(logits, idx, G.d_gates, G.d_logits, B.status, score=score, scale=scale,
                  flags=MOE_FLAG_NORMALIZE_GATES if normalize_gates else 0, stream=stream)
    if padding is not None:   # whatever their logits hold
        with on:
            G.d_logits.masked_fill_(padding[:, None], 0.0)
    return G


# --------------------------------------------- the layer on 8-bit integer experts
@dataclass
class Int8Operand:
    """8-bit integer weights, a scale for each output channel."""
    q: torch.Tensor       # [e, rows, cols] int8
    scale: torch.Tensor   # [e, rows] fp32


def quantize_weights_int8(w) -> Int8Operand:
    """8-bit form of expert weights [e, rows, cols] (bf16 or fp32), made once."""
    e, rows, cols = w.shape
    q = torch.empty((e, rows, cols), dtype=torch.int8, device=w.device)
    scale = torch.empty((e, rows), dtype=torch.float32, device=w.device)
    moe_quantize_rows_int8(w, q, scale, torch.zeros((1,), dtype=torch.int32, device=w.device))
    return Int8Operand(q, scale)


def run_layer_int8(x, logits, bias, w1: Int8Operand, b1, w3: Optional[Int8Operand], w2: Int8Operand, b2, act, k,
                   bufs: MoESortedBuffers, score="softmax", groups=1, topk_groups=1, group_top=1, scale=1.0,
                   normalize_gates=True, padding=None, stream=None):
    """run_layer_sorted with 8-bit integer experts (weights from
    quantize_weights_int8, buffers of alloc_layer_sorted with int8=True): the
    tokens are quantised straight into their rows."""
    B = bufs
    w3 = w3 or Int8Operand(None, None)
    _route_sorted(B, logits, bias, k, score, groups, topk_groups, group_top, scale, normalize_gates, padding, stream)
    moe_quantize_rows_int8(x, B.xs_q, B.xs_scale, B.status, rows=B.rows, stream=stream)
    moe_expert_ffn_int8(B.xs_q, B.xs_scale, B.offsets, w1.q, w1.scale, b1, w3.q, w3.scale, w2.q, w2.scale, b2, act,
                        B.ffn_ws, B.out, B.status, stream=stream)
    moe_decode_sorted(B.out, B.rows, B.y, B.status, gates=B.gates, stream=stream)
    return B.y
