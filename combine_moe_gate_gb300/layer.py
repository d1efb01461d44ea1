"""Device buffers for one MoE layer forward, allocated with torch (plumbing only).

The layer itself runs in libmoe_gate.so (`moe_layer_forward`, or the single
calls that `run_layer_fp4` makes); this module sizes and allocates the tensors
the C ABI writes into.
"""

from dataclasses import dataclass
from typing import Optional

import torch

from . import (MOE_BF16, MOE_F32, MOE_FLAG_NORMALIZE_GATES, moe_capacity_bound,
               moe_capacity_locations, moe_capacity_workspace_size, moe_decode, moe_encode,
               moe_expert_ffn_fp4, moe_expert_ffn_fp4_workspace_size, moe_fp4_scale_bytes,
               moe_layer_forward, moe_layer_forward_host, moe_layer_workspace_size,
               moe_quantize_fp4, moe_route_topk)


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
