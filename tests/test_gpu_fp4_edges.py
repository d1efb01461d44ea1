"""The 4-bit operands at the ends of their ranges."""

import numpy as np
import pytest
import torch

import combine_moe_gate_gb300 as M

from test_gpu_fp4 import data, dequant, quant, quantize64, unpack, untile
from test_gpu_fp4_tiles import check_hidden, ffn, untiled, values

pytestmark = pytest.mark.gpu


# Both sides of the ranges in which the quantiser takes the short forms of the
# division (6 g within 2^-40 .. 2^40, block maxima within 2^-60 .. 2^60).
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lg", [-100, -60, -50, -43, -42, -41, -20, 0, 20, 37, 38, 50, 60, 100])
def test_factors_over_their_range_are_bit_exact(lg, dt):
    g = torch.tensor([1.37 * 2.0 ** lg, 2.0 ** lg], dtype=torch.float32, device="cuda")
    x = data((2, 40, 512), 91 + lg, torch.float32)
    # rows from far below the smallest scale to beyond the largest
    x *= torch.exp2(torch.linspace(-14, 12, 40, device="cuda"))[None, :, None] * 2.0 ** min(lg, 100)
    x = x.clamp(-3e38, 3e38).to(dt)
    q, sc = quant(x, "nv", g)
    back = dequant(q, sc, "nv", g=g).cpu().numpy()
    for j in range(2):
        qo, so, vo = quantize64(x[j].float().cpu().numpy(), "nv", g[j].item())
        assert np.array_equal(untile(sc[j].cpu().numpy(), 40, 32), so)
        assert np.array_equal(unpack(q[j].cpu().numpy()), qo)
        assert np.array_equal(back[j], vo)


@pytest.mark.parametrize("scale", [2.0 ** 60, 2.0 ** -60])
def test_block_maxima_at_the_switch_are_bit_exact(scale):
    x = data((1, 64, 512), 97, torch.float32)
    x = x / x.abs().amax(2, keepdim=True) * torch.linspace(0.98, 1.02, 64, device="cuda")[None, :, None] * scale
    for lg in (20, 30, 39, -25, -39):
        g = torch.tensor([2.0 ** lg * 1.1], device="cuda")
        q, sc = quant(x, "nv", g)
        qo, so, _ = quantize64(x[0].cpu().numpy(), "nv", g[0].item())
        assert np.array_equal(untile(sc[0].cpu().numpy(), 64, 32), so)
        assert np.array_equal(unpack(q[0].cpu().numpy()), qo)


def test_scales_without_a_reciprocal_give_zeros():
    """A factor so small that 1 / (s8 g) overflows fp32: the codes are 0, those of
    zeros too; the first factors whose scales have a reciprocal are exact."""
    for lg, tiny in ((-124, False), (-126, False), (-132, True), (-140, True), (-149, True)):
        g = torch.tensor([2.0 ** lg], dtype=torch.float32, device="cuda")
        x = torch.zeros((1, 3, 64), device="cuda")
        # blocks with s8 = 1 (the largest is 6 g), and one with zeros between
        x[0, 0] = 6.0 * 2.0 ** lg * torch.tensor([1.0, -1.0, 0.5, 0.0], dtype=torch.float64).repeat(16).float().cuda()
        x[0, 1, ::16] = 6.0 * 2.0 ** lg
        q, sc = quant(x, "nv", g)
        codes, tiles = unpack(q[0].cpu().numpy()), untile(sc[0].cpu().numpy(), 3, 4)
        assert (tiles[:2] == 0x38).all() and (tiles[2] == 0).all()
        if tiny:
            assert (codes & 7 == 0).all()
            assert (dequant(q, sc, "nv", g=g) == 0).all()
        else:
            qo, _, _ = quantize64(x[0].cpu().numpy(), "nv", g[0].item())
            assert np.array_equal(codes, qo)


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_a_bad_weight_spoils_its_own_block_only(bad):
    w = data((3, 40, 128), 95) * 0.02
    clean = M.quantize_weights_fp4(w, "nv")
    w[1, 7, 33] = bad
    op = M.quantize_weights_fp4(w, "nv")
    torch.cuda.synchronize()
    # expert 1's factor is still that of its finite values
    finite = torch.where(torch.isfinite(w), w, torch.zeros_like(w)).float().abs().amax((1, 2)) / (6.0 * 448.0)
    assert torch.equal(op.global_scale, finite)
    v, ref = (dequant(o.q, o.scale, "nv", g=o.global_scale) for o in (op, clean))
    assert bool(torch.isnan(v[1, 7, 32:48]).all())
    v[1, 7, 32:48] = ref[1, 7, 32:48]
    assert bool(torch.isfinite(v).all()) and torch.equal(v[0], ref[0]) and torch.equal(v[2], ref[2])
    w[1, 7, 33] = 0
    # (block errors: half an e2m1 step of 6 with a scale within 2^-4, and the e4m3 scale's own)
    assert bool(((v - w.float()).abs() <= 0.2 * w.float().abs().amax((1, 2), keepdim=True)).all())


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
