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


# ------------------------------------------- several tiles per CTA pair
# At least three tiles for each of the 76 pairs of the chip, so that both
# accumulators, their overlap and every barrier phase are used and used again;
# several K stages, ragged counts, widths that end inside a tile.
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
MANY = dict(e=5, c_max=1030, c=1029, k=1056, n=4128, kept=[1030, 641, 0, 1029, 300])


def tiles(kept, c, width, tile):
    return sum(-(-min(r, c) // 256) for r in kept) * -(-width // tile)


def values(q, sc, fmt, g, j):
    """64-bit values of expert j's rows: code * scale is exact in fp32, the factor is applied in 64 bits."""
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    v = torch.empty((1, q.shape[1], 2 * q.shape[2]), device="cuda")
    M.moe_dequantize_fp4(q[j:j + 1], sc[j:j + 1], fmt, v, st)
    return v[0].double() * (1.0 if g is None else g[j].item())


def product_bound(mag, want, k):
    """One bf16 rounding and k fp32 additions of products whose magnitudes sum to mag."""
    return 2.0 ** -8 * want.abs() + 2.0 ** -23 * (k + 8) * mag + 1e-30


def check_rows(out, j, r, hid, w, bias, k):
    want, mag = hid @ w.t(), hid.abs() @ w.abs().t()
    if bias is not None:
        want = want + bias.double()
    err = (out[j, :r].double() - want).abs()
    assert bool((err <= product_bound(mag, want, k)).all()), (j, err.max().item())
    assert bool((out[j, r:] == -9.0).all())


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("use_bias", [False, True])
def test_product_over_many_tiles(fmt, use_bias):
    e, c_max, c, k, n, kept = (MANY[x] for x in ("e", "c_max", "c", "k", "n", "kept"))
    assert tiles(kept, c, n, 256) >= 3 * 76
    ga, gb = factors(e, fmt, 1, 0.005), factors(e, fmt, 2, 0.003)
    a, b = quant(data((e, c_max, k), 71), fmt, ga), quant(data((e, n, k), 72), fmt, gb)
    bias = data((e, n), 73) if use_bias else None
    counts, c_dev = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (kept, [c]))
    outs = []
    for _ in range(3):
        out = torch.full((e, c_max, n), -9.0, dtype=torch.bfloat16, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        M.moe_product_fp4(*a, ga, counts, c_dev, *b, gb, bias, fmt, out, st)
        torch.cuda.synchronize()
        status_ok(st)
        outs.append(out)
    assert all(torch.equal(o, outs[0]) for o in outs[1:])
    for j in range(e):
        r = min(kept[j], c)
        check_rows(outs[0], j, r, values(*a, fmt, ga, j)[:r], values(*b, fmt, gb, j),
                   None if bias is None else bias[j], k)


def untiled(sc, rows, blocks):
    """Scale bytes [rows, blocks] of one expert's tiles, and those past the last block."""
    nt = -(-blocks // 4)
    r, b = torch.arange(rows, device="cuda")[:, None], torch.arange(4 * nt, device="cuda")[None]
    s = sc[((r // 128) * nt + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4]
    return s[:, :blocks].long(), s[:, blocks:]


def scale_values(code, fmt):
    if fmt == "mx":
        return torch.ldexp(torch.ones_like(code, dtype=torch.float64), code - 127)
    ex, man = code >> 3, (code & 7).double()
    return torch.where(ex > 0, torch.ldexp(8 + man, ex - 10), man * 2.0 ** -9)


def check_hidden(hid, tol, hv, code, fmt, g):
    """Whether the codes hv (values) with scale bytes `code` stand for the
    quantisation of some numbers within tol of hid: the scale lies between those of
    the block's largest magnitude less and plus its tolerance, and each value is no
    further from its code than half the gap there, plus its tolerance."""
    blk = 32 if fmt == "mx" else 16
    rows = hid.shape[0]
    amax, t = hid.abs().view(rows, -1, blk).amax(2), tol.view(rows, -1, blk).amax(2)
    s = scale_values(code, fmt)
    if fmt == "mx":
        # s <= amax / 4 < 2 s up to the tolerance; 1 for a block of zeros
        ok = (4 * s <= amax + t) & (amax - t < 8 * s)
        ok |= (amax <= t) & (code == 127)
    else:
        # within half an e4m3 step (2^-4 relative, 2^-10 below 2^-6) of amax / (6 g), at most 448
        x, dx = amax / (6 * g), t / (6 * g) + 1e-6 * amax / (6 * g)
        ok = ((s - x).abs() <= 2.0 ** -4 * s + 2.0 ** -10 + dx) | ((s == 448) & (x + dx >= 448))
        s = s * g
    assert bool(ok.all())
    s = s.repeat_interleave(blk, 1)
    grid = torch.tensor(E2M1, device="cuda", dtype=torch.float64)
    y = torch.where(s > 0, hv.abs() / s, torch.zeros_like(s))
    at = torch.searchsorted(grid, (y - 0.01).contiguous())   # y is on the grid up to rounding
    up = torch.where(at == 7, torch.inf, (grid[(at + 1).clamp(max=7)] - grid[at]) / 2)
    down = torch.where(at == 0, 0.25, (grid[at] - grid[(at - 1).clamp(min=0)]) / 2)
    d = torch.where(hv < 0, -hid, hid) - hv.abs()
    slack = tol + 1e-6 * s
    assert bool((((d <= up * s + slack) & (-d <= down * s + slack)) | (s == 0)).all())


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("act", ["relu", "gelu", "swiglu"])
def test_ffn_over_many_tiles(fmt, act):
    e, c_max, c, m, h, kept = (MANY[x] for x in ("e", "c_max", "c", "k", "n", "kept"))
    swiglu = act == "swiglu"
    assert tiles(kept, c, h, 128 if swiglu else 256) >= 3 * 76
    xs, gh, w, b = operands(fmt, act, e, c_max, m, h, 81)
    counts = torch.tensor(kept, dtype=torch.int32, device="cuda")
    out, ws = ffn(fmt, act, xs, gh, w, b, counts, c, fill=0x55)
    again, _ = ffn(fmt, act, xs, gh, w, b, counts, c, fill=0x33)
    assert torch.equal(out, again)
    nq = e * c_max * h // 2
    hq = ws[:nq].view(e, c_max, h // 2)
    at = (nq + 255) // 256 * 256
    hs = ws[at:at + e * M.moe_fp4_scale_bytes(fmt, c_max, h)].view(e, -1)
    for j in range(e):
        r = min(kept[j], c)
        assert bool((hq[j, r:] == 0x55).all())
        if r == 0:
            assert bool((out[j] == -9.0).all())
            continue
        x, w1 = values(*xs[:2], fmt, xs[2], j)[:r], values(*w[0][:2], fmt, w[0][2], j)
        pre = x @ w1.t()
        tol = 2.0 ** -23 * (m + 16) * (x.abs() @ w1.abs().t()) + 1e-6 * pre.abs()
        if swiglu:
            w3 = values(*w[1][:2], fmt, w[1][2], j)
            up = x @ w3.t()
            tol_up = 2.0 ** -23 * (m + 16) * (x.abs() @ w3.abs().t()) + 1e-6 * up.abs()
            sg = torch.sigmoid(pre)
            hid = pre * sg * up   # |silu'| <= 1.1
            tol = 1.1 * tol * up.abs() + (pre * sg).abs() * tol_up + 1e-6 * hid.abs()
        else:
            b1 = b[0][j].double()
            pre = pre + b1
            hid = torch.relu(pre) if act == "relu" else torch.nn.functional.gelu(pre)
            # |gelu'| <= 1.13, its own error below 1e-6 of |pre|
            tol = 1.2 * (tol + 2.0 ** -23 * b1.abs()) + 1e-6 * pre.abs()
        code, rest = untiled(hs[j], r, h // (32 if fmt == "mx" else 16))
        assert bool((rest == 0).all())
        hv = values(hq, hs, fmt, gh, j)[:r]
        check_hidden(hid, tol, hv, code, fmt, 1.0 if gh is None else gh[j].item())
        check_rows(out, j, r, hv, values(*w[2][:2], fmt, w[2][2], j), None if b[1] is None else b[1][j], h)
