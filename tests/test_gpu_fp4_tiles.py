"""The 4-bit products where a CTA pair works through several tiles, or where one
of its producers falls behind."""

import pytest
import torch

import combine_moe_gate_gb300 as M

from gpu_util import status_ok
from test_gpu_fp4 import data, factors, quant

pytestmark = pytest.mark.gpu


def operands(fmt, act, e, c_max, m, h, seed):
    """Quantised input, weights (w1, w3, w2), factors and biases of an expert FFN."""
    swiglu = act == "swiglu"
    g = [factors(e, fmt, seed + i, s) for i, s in enumerate((0.004, 0.05, 0.002, 0.002, 0.002))]
    x = data((e, c_max, m), seed)
    w = [data((e, h, m), seed + 1), data((e, h, m), seed + 2) if swiglu else None, data((e, m, h), seed + 3)]
    q = [(None, None, None) if t is None else (*quant(t, fmt, f), f) for t, f in zip(w, g[2:])]
    b = (None, None) if swiglu else (data((e, h), seed + 4), data((e, m), seed + 5))
    return (*quant(x, fmt, g[0]), g[0]), g[1], q, b


def ffn(fmt, act, xs, gh, w, b, counts, c, fill=0):
    """out and the workspace (codes and scales of the hidden) of one call."""
    e, c_max, m = xs[0].shape[0], xs[0].shape[1], 2 * xs[0].shape[2]
    h = w[0][0].shape[1]
    ws = torch.full((M.moe_expert_ffn_fp4_workspace_size(fmt, act, e, c_max, m, h),), fill, dtype=torch.uint8,
                    device="cuda")
    out = torch.full((e, c_max, m), -9.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.moe_expert_ffn_fp4(*xs, gh, counts, torch.tensor([c], dtype=torch.int32, device="cuda"), *w[0], b[0], *w[1],
                         *w[2], b[1], fmt, act, ws, out, st)
    torch.cuda.synchronize()
    status_ok(st)
    return out, ws


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("act", ["swiglu", "relu"])
def test_a_producer_without_copies_may_fall_behind(fmt, act):
    """Tiles whose rows all lie in the first CTA of the pair give the second CTA's
    A producers nothing to copy; held back by 20 us a stage they must still keep in
    step with a ring that is otherwise ten times as fast."""
    e, c_max, m, h = 3, 300, 4096, 2080
    counts = torch.tensor([16, 300, 100], dtype=torch.int32, device="cuda")
    args = operands(fmt, act, e, c_max, m, h, 61)
    want, _ = ffn(fmt, act, *args, counts, c_max)
    M.moe_debug_lag_gemms(2)
    try:
        got, _ = ffn(fmt, act, *args, counts, c_max)
    finally:
        M.moe_debug_lag_gemms(0)
    assert torch.equal(got, want) and bool(torch.isfinite(want[0, :16].float()).all())
