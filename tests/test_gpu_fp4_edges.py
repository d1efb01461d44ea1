"""The 4-bit operands at the ends of their ranges."""

import pytest
import torch

import combine_moe_gate_gb300 as M

from test_gpu_fp4 import data, quant
from test_gpu_fp4_tiles import check_hidden, ffn, untiled, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_gelu_over_its_range(fmt):
    """Hidden values of prescribed pre-activations, in blocks of like magnitude (a
    tail's blocks are scaled by the tail): bias + one small product a row.

    The value's own error: 2e-5 of it down to -6 and 4e-4 down to -8, plus 2e-7 of
    |pre| on the other side of zero; and fp32's rounding of the pre-activation,
    2^-24 |pre| times the slope, which in the tail is at most (|pre| + 1) |GELU|."""
    e, rows, m = 32, 8, 32
    b = torch.cat((-torch.logspace(-3, 3, 1536, base=2.0, dtype=torch.float64).flip(0),
                   torch.logspace(-6, 3, 512, base=2.0, dtype=torch.float64))).to(torch.bfloat16)
    h = b.numel()
    x, w1, w2 = torch.zeros((e, rows, m), device="cuda"), torch.zeros((e, h, m), device="cuda"), data((e, m, h), 3)
    x[:, :, 0] = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    if fmt == "mx":
        g = gw = gh = None
        w1[:, :, 0] = 2.0 ** -9                               # both exact in MX
    else:
        g = torch.ones(e, device="cuda")
        x[:, :, 1] = 6.0                                      # (w1 is 0 there:) block scales of 1, codes are the values
        gw = (torch.linspace(0.0, 1.0, e) * 2.0 ** -9 + 1e-6).cuda()
        w1[:, :, 0] = 6.0 * gw[:, None]                       # block scales of 1, code 6
        gh = torch.exp2(-torch.arange(e) * 1.25 - 12).float().cuda()
    xq, wq = quant(x, fmt, g), quant(w1, fmt, gw)
    counts = torch.full((e,), rows, dtype=torch.int32, device="cuda")
    bias = b[None].expand(e, h).contiguous().cuda()
    out, ws = ffn(fmt, "gelu", (*xq, g), gh, [(*wq, gw), (None, None, None), (*quant(w2, fmt), None)], (bias, None),
                  counts, rows)
    nq = e * rows * h // 2
    hq = ws[:nq].view(e, rows, h // 2)
    at = (nq + 255) // 256 * 256
    hs = ws[at:at + e * M.moe_fp4_scale_bytes(fmt, rows, h)].view(e, -1)
    for j in range(e):
        pre = values(*xq, fmt, g, j) @ values(*wq, fmt, gw, j).t() + b.double().cuda()
        val = 0.5 * pre * torch.erfc(-pre * 0.5 ** 0.5)
        own = torch.where(pre < -6.0, 4e-4, 2e-5) * val.abs() + torch.where(pre > 0, 2e-7 * pre, torch.zeros_like(pre))
        tol = own + 2.0 ** -24 * pre.abs() * torch.where(pre < 0, (pre.abs() + 1) * val.abs(), torch.full_like(val, 1.13))
        code, _ = untiled(hs[j], rows, h // (32 if fmt == "mx" else 16))
        check_hidden(val, tol, values(hq, hs, fmt, gh, j), code, fmt, 1.0 if gh is None else gh[j].item())
