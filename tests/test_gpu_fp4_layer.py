"""The 4-bit layer end to end, and what the operators must survive: pointers that
are only 16-byte aligned, offsets beyond 32 bits, a stream of their own, a GEMM
whose wait runs out."""

import time

import numpy as np
import pytest
import torch

import combine_moe_gate_gb300 as M

from gpu_util import bits, status_ok
from test_gpu_fp4 import act64, data, dequant, quant, quantize64, values64
from test_gpu_route import scores64

pytestmark = pytest.mark.gpu


def q64(x, fmt, g):
    return quantize64(np.ascontiguousarray(x, np.float32), fmt, g)[2].astype(np.float64)


@pytest.mark.parametrize("fmt,act,score", [("nv", "swiglu", "sigmoid"), ("mx", "gelu", "softmax"), ("nv", "relu", "softmax")])
@pytest.mark.parametrize("s,f", [(1, 0.0), (200, 1.0), (333, 0.0)])
def test_layer_matches_64_bit(fmt, act, score, s, f):
    m, e, k, h = 256, 16, 4, 160
    swiglu = act == "swiglu"
    x, logits = data((s, m), 41), data((s, e), 42, torch.float32)
    bias = (torch.randn(e, generator=torch.Generator().manual_seed(1)) * 0.05).cuda()
    w = [data((e, h, m), 43), data((e, h, m), 44) if swiglu else None, data((e, m, h), 45)]
    b1, b2 = (None, None) if swiglu else (data((e, h), 46), data((e, m), 47))
    ops = [None if t is None else M.quantize_weights_fp4(t, fmt) for t in w]
    gx = torch.full((e,), 0.013, device="cuda") if fmt == "nv" else None
    gh = torch.full((e,), 0.11, device="cuda") if fmt == "nv" else None
    bufs = M.alloc_layer_fp4(s, m, e, k, h, act, fmt, f)
    kw = dict(buf_global=gx, hid_global=gh, score=score, groups=4, topk_groups=2, group_top=2, scale=2.5)
    y = M.run_layer_fp4(x, logits, bias, ops[0], b1, ops[1], ops[2], b2, fmt, act, k, f, bufs, **kw)
    torch.cuda.synchronize()
    status_ok(bufs.status)
    idx, loc = bufs.idx.cpu().numpy(), bufs.loc.cpu().numpy()
    gates, c = bufs.gates.cpu().numpy().astype(np.float64), int(bufs.c_dev.item())
    # the gates are the chosen scores over their sum, times the scale
    sc = np.take_along_axis(scores64(logits.cpu().numpy().astype(np.float64), score), idx.T, 1)
    assert np.allclose(gates.T, 2.5 * sc / sc.sum(1, keepdims=True), rtol=1e-5, atol=0)
    wv = [None if o is None else values64(o.q, o.scale, fmt, o.global_scale) for o in ops]
    xv = q64(x.float().cpu().numpy(), fmt, 0.013 if fmt == "nv" else 1.0)
    want = np.zeros((s, m))
    dropped = 0
    for r in range(k):
        for t in range(s):
            j = idx[r, t]
            if loc[r, t] >= c:
                dropped += 1
                continue
            hid = wv[0][j] @ xv[t]
            if swiglu:
                hid = hid / (1 + np.exp(-hid)) * (wv[1][j] @ xv[t])
            else:
                hid = act64(hid + b1[j].float().cpu().numpy().astype(np.float64), act)
            hv = q64(hid[None], fmt, 0.11 if fmt == "nv" else 1.0)[0]
            o = wv[2][j] @ hv
            if b2 is not None:
                o = o + b2[j].float().cpu().numpy()
            want[t] += gates[r, t] * o
    assert (dropped > 0) == (f > 0 and s > 1)
    got = y.float().cpu().numpy()
    # two bf16 roundings (2^-9 each) and the few hidden codes that fp32 rounds the other way
    assert np.linalg.norm(got - want) <= 6e-3 * np.linalg.norm(want)
    # the same on a stream of its own, bit for bit
    side = torch.cuda.Stream()
    again = M.alloc_layer_fp4(s, m, e, k, h, act, fmt, f)
    side.wait_stream(torch.cuda.current_stream())
    M.run_layer_fp4(x, logits, bias, ops[0], b1, ops[1], ops[2], b2, fmt, act, k, f, again, stream=side, **kw)
    side.synchronize()
    assert torch.equal(again.y, y) and torch.equal(again.idx, bufs.idx)


def shifted(t, by):
    """A copy of t that starts `by` bytes past a 256-byte boundary."""
    raw = torch.empty(t.numel() * t.element_size() + 256, dtype=torch.uint8, device="cuda")
    v = raw[by:by + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
    v.copy_(t)
    assert v.data_ptr() % 32 == by % 32
    return v


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_buffers_on_16_byte_boundaries(fmt, dt):
    x = data((2, 130, 672), 5, dt)
    q, sc = quant(x, fmt)
    q2, sc2 = quant(shifted(x, 16), fmt)
    assert torch.equal(q, q2)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q3, sc3 = shifted(torch.zeros_like(q), 16), shifted(sc, 16)
    M.moe_quantize_fp4(x, fmt, q3, sc3, st)
    want = dequant(q, sc, fmt, dt)
    out = shifted(torch.zeros_like(x), 16)
    M.moe_dequantize_fp4(q3, sc3, fmt, out, st)
    torch.cuda.synchronize()
    status_ok(st)
    assert torch.equal(q3, q) and torch.equal(out, want)
    w = data((2, 48, 672), 6)
    wq, wsc = quant(w, fmt)
    cnt = torch.tensor([130, 77], dtype=torch.int32, device="cuda")
    cd = torch.tensor([130], dtype=torch.int32, device="cuda")
    bias = data((2, 48), 7)
    a = torch.zeros((2, 130, 48), dtype=torch.bfloat16, device="cuda")
    b = shifted(a, 16)
    M.moe_product_fp4(q, sc, None, cnt, cd, wq, wsc, None, bias, fmt, a, st)
    M.moe_product_fp4(q3, sc3, None, cnt, cd, shifted(wq, 16), shifted(wsc, 16), None, shifted(bias, 16), fmt, b, st)
    torch.cuda.synchronize()
    status_ok(st)
    assert torch.equal(a, b) and a.abs().sum() > 0


def test_offsets_beyond_32_bits():
    """Rows whose first element lies past 2^31: the last ones must be right."""
    rows, cols, tail = 70000, 32768, 130
    x = torch.zeros((1, rows, cols), dtype=torch.bfloat16, device="cuda")
    x[0, -tail:] = data((tail, cols), 3)
    q, sc = quant(x, "nv")
    ref_q, _ = quant(x[:, -tail:].contiguous(), "nv")
    assert torch.equal(q[:, -tail:], ref_q)
    back = dequant(q, sc, "nv", torch.bfloat16)
    assert torch.equal(back[:, -tail:], dequant(*quant(x[:, -tail:].contiguous(), "nv"), "nv", torch.bfloat16))
    del x, back, q, sc
    # a product whose output has more than 2^31 elements
    k = 64
    a = torch.zeros((1, rows, k), dtype=torch.bfloat16, device="cuda")
    a[0, -tail:] = data((tail, k), 4)
    w = data((1, cols, k), 5)
    aq, asc = quant(a, "mx")
    wq, wsc = quant(w, "mx")
    cd = torch.tensor([rows], dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((1, rows, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    M.moe_product_fp4(aq, asc, None, cd, cd, wq, wsc, None, None, "mx", out, st)
    torch.cuda.synchronize()
    status_ok(st)
    av = dequant(aq, asc, "mx")[0, -tail:].double()
    wv = dequant(wq, wsc, "mx")[0].double()
    want = av @ wv.t()
    mag = av.abs() @ wv.abs().t()
    err = (out[0, -tail:].double() - want).abs()
    assert bool((err <= 2.0 ** -8 * want.abs() + 2.0 ** -23 * (k + 8) * mag).all())
    assert bool((out[0, :-tail] == 0).all())


def test_router_offsets_beyond_32_bits():
    s, e = (1 << 31) // 512 + 1000, 512
    x = torch.zeros((s, e), dtype=torch.bfloat16, device="cuda")
    hot = torch.arange(s, device="cuda") * 7 % e
    x.scatter_(1, hot[:, None], 1.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    idx = torch.empty((1, s), dtype=torch.int32, device="cuda")
    gates = torch.empty((1, s), device="cuda")
    M.moe_route_topk(x, None, 1, idx, gates, st, score="sigmoid")
    d = torch.empty((s, e), dtype=torch.bfloat16, device="cuda")
    M.moe_route_bwd(x, idx, torch.ones_like(gates), d, st, score="sigmoid")
    torch.cuda.synchronize()
    status_ok(st)
    assert bool((idx[0] == hot).all()) and bool((gates == gates[0, 0]).all())
    g = torch.sigmoid(torch.ones((), dtype=torch.float64)).item()
    assert abs(gates[0, -1].item() - g) < 1e-6
    assert bool((d[-1000:].gather(1, hot[-1000:, None]).double() - g * (1 - g)).abs().max() < 1e-3)
    assert bool((d[-1000:].count_nonzero(1) == 1).all())


def test_fp4_gemm_bounded_wait_runs_out_and_the_context_stays_usable():
    e, c_max, m, h = 2, 256, 256, 512
    x, w1, w2 = data((e, c_max, m), 1), data((e, h, m), 2), data((e, m, h), 3)
    q = [quant(t, "nv") for t in (x, w1, w2)]
    cnt = torch.tensor([200, 131], dtype=torch.int32, device="cuda")
    cd = torch.tensor([c_max], dtype=torch.int32, device="cuda")
    ws = torch.zeros(M.moe_expert_ffn_fp4_workspace_size("nv", "gelu", e, c_max, m, h), dtype=torch.uint8, device="cuda")

    def run(out):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        M.moe_expert_ffn_fp4(*q[0], None, None, cnt, cd, *q[1], None, None, None, None, None, *q[2], None, None, "nv",
                             "gelu", ws, out, st)
        torch.cuda.synchronize()
        return int(st.item())

    ref = torch.zeros((e, c_max, m), dtype=torch.bfloat16, device="cuda")
    assert run(ref) == M.MOE_OK
    M.moe_debug_stall_gemms(1)
    try:
        stalled = torch.full((e, c_max, m), -5.0, dtype=torch.bfloat16, device="cuda")
        t0 = time.monotonic()
        code = run(stalled)
        dt = time.monotonic() - t0
    finally:
        M.moe_debug_stall_gemms(0)
    assert code == M.MOE_ERR_TIMEOUT, M.status_str(code)
    assert 0.5 < dt < 30.0, dt
    assert bool((stalled == -5.0).all())
    again = torch.zeros_like(ref)
    assert run(again) == M.MOE_OK and (bits(again) == bits(ref)).all()
