"""The microscaled 4-bit operands on the GPU: the quantiser and the expander bit
for bit against a plain 64-bit form, the products and the FFN step by step
within bounds of their fp32 accumulation and final rounding."""

import numpy as np
import pytest
import torch

import combine_moe_gate_gb300 as M

from gpu_util import status_ok

pytestmark = pytest.mark.gpu

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
BLK = {"mx": 32, "nv": 16}
E4M3 = np.array([m / 8 * 2.0 ** -6 if ex == 0 else (1 + m / 8) * 2.0 ** (ex - 7)
                 for ex in range(16) for m in range(8)][:127])


def nearest(v, grid):
    """Index of the nearest grid value, ties to the even index, v >= 0 and <= grid[-1]."""
    hi = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
    lo = hi - 1
    up, down = grid[hi] - v, v - grid[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def quantize64(x, fmt, g):
    """fp32 x [rows, cols] -> codes [rows, cols], scale codes [rows, blocks], values.
    Each step that the format defines in fp32 is rounded to fp32 once."""
    f32 = np.float32
    b = BLK[fmt]
    v = x.reshape(x.shape[0], -1, b).astype(np.float64)
    amax = np.abs(v).max(2)
    if fmt == "mx":
        _, ex = np.frexp(np.where(amax > 0, amax, 1.0))
        sc = np.where(amax > 0, np.maximum(ex - 1 - 2, -127), 0) + 127
        s = np.ldexp(1.0, sc - 127)
        inv = np.ldexp(1.0, 127 - sc)
    else:
        t = (amax.astype(f32) / f32(f32(6) * f32(g))).astype(np.float64)
        sc = nearest(np.minimum(t, 448.0), E4M3)
        s = (E4M3[sc].astype(f32) * f32(g)).astype(np.float64)
        with np.errstate(divide="ignore"):
            inv = np.where(s > 0, (f32(1) / s.astype(f32)).astype(np.float64), 0.0)
    y = (v * inv[..., None]).astype(f32).astype(np.float64)
    q = nearest(np.minimum(np.abs(y), 6.0), E2M1) + 8 * np.signbit(y)
    vals = (E2M1[q & 7] * s[..., None]).astype(f32) * np.where(q & 8, -1, 1)
    return q.reshape(x.shape).astype(np.uint8), sc.astype(np.uint8), vals.reshape(x.shape)


def untile(t, rows, blocks):
    nt = -(-blocks // 4)
    r, b = np.arange(rows)[:, None], np.arange(nt * 4)[None]
    return t[((r // 128) * nt + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4]


def unpack(q):
    return np.stack([q & 15, q >> 4], -1).reshape(q.shape[0], 2 * q.shape[1])


def quant(x, fmt, g=None, counts=None, c_dev=None):
    b, r, c = x.shape
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = torch.full((b, r, c // 2), 0xAA, dtype=torch.uint8, device="cuda")
    sc = torch.full((b, M.moe_fp4_scale_bytes(fmt, r, c)), 0x55, dtype=torch.uint8, device="cuda")
    M.moe_quantize_fp4(x, fmt, q, sc, st, global_scale=g, counts=counts, c_dev=c_dev)
    torch.cuda.synchronize()
    status_ok(st)
    return q, sc


def dequant(q, sc, fmt, dt=torch.float32, g=None, counts=None, c_dev=None):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((q.shape[0], q.shape[1], 2 * q.shape[2]), -5.0, dtype=dt, device="cuda")
    M.moe_dequantize_fp4(q, sc, fmt, out, st, global_scale=g, counts=counts, c_dev=c_dev)
    torch.cuda.synchronize()
    status_ok(st)
    return out


def data(shape, seed, dt=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(torch.randn(shape[:-1] + (1,), generator=g))
    return x.to(dt).cuda()


SHAPES = [(1, 1, 32), (1, 37, 96), (3, 50, 64), (2, 130, 160), (1, 129, 2080), (1, 5, 16416), (2, 300, 512)]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_quantize_is_bit_exact(fmt, dt, shape):
    b, r, c = shape
    x = data(shape, c + r, dt)
    x[0, 0, :32] = 0                               # blocks of zeros
    if r > 4:
        x[0, 1] *= 1e-30                           # NV: scales that underflow to 0
        x[0, 2] = 2.0 ** -130                      # subnormal values
        x[0, 3, 5] = -3e38                         # the widest range in one block
        x[0, 4, ::2] = 0.75                        # ties
        x[0, 4, 1::2] = 6.0
    g = torch.rand(b, generator=torch.Generator().manual_seed(1)).add_(0.5).mul_(0.01).cuda() if fmt == "nv" else None
    q, sc = quant(x, fmt, g)
    back = dequant(q, sc, fmt, g=g).cpu().numpy()
    half = dequant(q, sc, fmt, torch.bfloat16, g=g).cpu()
    for j in range(b):
        qo, so, vo = quantize64(x[j].float().cpu().numpy(), fmt, 1.0 if g is None else g[j].item())
        tiles = untile(sc[j].cpu().numpy(), r, c // BLK[fmt])
        n = c // BLK[fmt]
        assert np.array_equal(tiles[:, :n], so) and (tiles[:, n:] == 0).all()
        assert np.array_equal(unpack(q[j].cpu().numpy()), qo)
        assert np.array_equal(back[j], vo)
        assert torch.equal(half[j], torch.from_numpy(vo).to(torch.bfloat16))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_quantize_writes_kept_rows_only(fmt):
    e, c_max, m = 4, 150, 160
    x = data((e, c_max, m), 7)
    counts = torch.tensor([150, 0, 17, -3], dtype=torch.int32, device="cuda")
    c_dev = torch.tensor([140], dtype=torch.int32, device="cuda")
    q, sc = quant(x, fmt, None, counts, c_dev)
    out = dequant(q, sc, fmt, g=None, counts=counts, c_dev=c_dev).cpu().numpy()
    n = m // BLK[fmt]
    for j, kept in enumerate([140, 0, 17, 0]):
        qo, so, vo = quantize64(x[j].float().cpu().numpy(), fmt, 1.0)
        tiles = untile(sc[j].cpu().numpy(), c_max, n)
        qn = q[j].cpu().numpy()
        assert np.array_equal(unpack(qn[:kept]), qo[:kept]) and (qn[kept:] == 0xAA).all()
        assert np.array_equal(tiles[:kept, :n], so[:kept]) and (tiles[kept:] == 0x55).all()
        assert np.array_equal(out[j, :kept], vo[:kept]) and (out[j, kept:] == -5.0).all()


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_blocks_with_infinity_or_nan_become_nan(fmt):
    x = data((1, 4, 128), 11)
    x[0, 0, 3] = float("inf")
    x[0, 1, 40] = float("nan")
    x[0, 2, 127] = -float("inf")
    q, sc = quant(x, fmt)
    v = dequant(q, sc, fmt).cpu().numpy()[0]
    b = BLK[fmt]
    for r, c in ((0, 3), (1, 40), (2, 127)):
        blk = c // b
        assert np.isnan(v[r, blk * b:(blk + 1) * b]).all()
        v[r, blk * b:(blk + 1) * b] = 0
    assert np.isfinite(v).all()


def test_a_2d_tensor_is_one_batch():
    x = data((1, 40, 64), 3)
    q3, s3 = quant(x, "mx")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, sc = torch.empty_like(q3[0]), torch.empty_like(s3)
    M.moe_quantize_fp4(x[0], "mx", q, sc, st)
    torch.cuda.synchronize()
    assert torch.equal(q, q3[0]) and torch.equal(untile_t(sc), untile_t(s3))


def untile_t(sc):
    return torch.from_numpy(untile(sc[0].cpu().numpy(), 40, 2))


# ---------------------------------------------------------------- products
def values64(q, sc, fmt, g=None):
    """Codes and tiled scales -> 64-bit values per batch."""
    out = []
    for j in range(q.shape[0]):
        codes = unpack(q[j].cpu().numpy())
        n = codes.shape[1] // BLK[fmt]
        s = untile(sc[j].cpu().numpy(), codes.shape[0], n)[:, :n].astype(np.int64)
        s = np.ldexp(1.0, s - 127) if fmt == "mx" else E4M3[s]
        v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
        v = (v.reshape(codes.shape[0], n, -1) * s[..., None]).reshape(codes.shape)
        out.append(v if g is None else v * float(g[j]))
    return out


def factors(e, fmt, seed, size):
    if fmt == "mx":
        return None
    return (torch.rand(e, generator=torch.Generator().manual_seed(seed)) * size + size).cuda()


def bound(mag, want, k):
    """One bf16 rounding (2^-9 relative, with margin 2^-8) and k fp32 additions
    of products whose magnitudes sum to mag."""
    return 2.0 ** -8 * np.abs(want) + 2.0 ** -23 * (k + 8) * mag + 1e-30


PRODUCTS = [
    # e, c_max, k, n, kept, c, bias
    (1, 1, 32, 8, [1], 1, True),
    (1, 128, 256, 256, [128], 128, False),
    (1, 300, 320, 264, [300], 300, True),
    (3, 40, 96, 136, [40, 0, 7], 33, True),
    (2, 520, 1056, 520, [513, 260], 520, False),
    (4, 64, 4096, 64, [64, 1, 0, 33], 64, True),
    (2, 257, 2080, 1032, [257, 129], 257, True),
    (9, 16, 288, 392, [1, 16, 0, 2, 3, 0, 0, 9, 1], 16, False),
]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("c", PRODUCTS, ids=lambda c: f"e{c[0]}_c{c[1]}_k{c[2]}_n{c[3]}")
def test_product_matches_64_bit(fmt, c):
    e, c_max, k, n, kept, cap, use_bias = c
    a, b = data((e, c_max, k), 21 + k), data((e, n, k), 22 + n)
    ga, gb = factors(e, fmt, 1, 0.005), factors(e, fmt, 2, 0.003)
    counts = torch.tensor(kept, dtype=torch.int32, device="cuda")
    c_dev = torch.tensor([cap], dtype=torch.int32, device="cuda")
    # rows past the kept ones, codes and scales alike, hold what quant() filled them with
    aq, asc = quant(a, fmt, ga, counts, c_dev)
    bq, bsc = quant(b, fmt, gb)
    bias = data((e, n), 23) if use_bias else None
    out = torch.full((e, c_max, n), -9.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.moe_product_fp4(aq, asc, ga, counts, c_dev, bq, bsc, gb, bias, fmt, out, st)
    torch.cuda.synchronize()
    status_ok(st)
    got = out.float().cpu().numpy()
    bv = values64(bq, bsc, fmt, gb)
    for j in range(e):
        r = min(kept[j], cap)
        assert (got[j, r:] == -9.0).all()
        if r == 0:
            continue
        av = values64(aq[j:j + 1, :r], asc[j:j + 1], fmt, None if ga is None else ga[j:j + 1])[0]
        want = av @ bv[j].T
        mag = np.abs(av) @ np.abs(bv[j]).T
        if use_bias:
            want = want + bias[j].float().cpu().numpy()
        assert (np.abs(got[j, :r] - want) <= bound(mag, want, k)).all(), (j, np.abs(got[j, :r] - want).max())


def test_product_ignores_nan_scales_of_rows_past_the_kept():
    e, c_max, k, n = 2, 200, 512, 256
    a, b = data((e, c_max, k), 1), data((e, n, k), 2)
    counts = torch.tensor([5, 130], dtype=torch.int32, device="cuda")
    c_dev = torch.tensor([c_max], dtype=torch.int32, device="cuda")
    outs = []
    for fill in (0x00, 0x7F):
        q = torch.full((e, c_max, k // 2), 0x77, dtype=torch.uint8, device="cuda")
        sc = torch.full((e, M.moe_fp4_scale_bytes("nv", c_max, k)), fill, dtype=torch.uint8, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        M.moe_quantize_fp4(a, "nv", q, sc, st, counts=counts, c_dev=c_dev)
        bq, bsc = quant(b, "nv")
        out = torch.zeros((e, c_max, n), dtype=torch.bfloat16, device="cuda")
        M.moe_product_fp4(q, sc, None, counts, c_dev, bq, bsc, None, None, "nv", out, st)
        torch.cuda.synchronize()
        status_ok(st)
        outs.append(out)
    assert torch.isfinite(outs[1].float()).all() and torch.equal(outs[0], outs[1])


# --------------------------------------------------------------------- FFN
def act64(v, act):
    if act == "relu":
        return np.maximum(v, 0.0)
    erf = torch.erf(torch.from_numpy(v) * 0.5 ** 0.5).numpy()
    return 0.5 * v * (1.0 + erf)


FFNS = [
    # e, c_max, m, h, act, kept, c
    (1, 1, 32, 32, "relu", [1], 1),
    (4, 64, 64, 160, "relu", [64, 0, 31, 40], 64),
    (3, 300, 256, 416, "gelu", [300, 0, 129], 290),
    (2, 260, 288, 96, "swiglu", [7, 260], 260),
    (2, 140, 1056, 544, "swiglu", [140, 1], 140),
    (3, 16, 2048, 1024, "gelu", [1, 16, 3], 16),
    (1, 515, 512, 768, "swiglu", [515], 515),
]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("c", FFNS, ids=lambda c: f"e{c[0]}_c{c[1]}_m{c[2]}_h{c[3]}_{c[4]}")
def test_expert_ffn_matches_64_bit(fmt, c):
    e, c_max, m, h, act, kept, cap = c
    swiglu = act == "swiglu"
    x = data((e, c_max, m), 31)
    w = [data((e, h, m), 32), data((e, h, m), 33) if swiglu else None, data((e, m, h), 34)]
    b1, b2 = (None, None) if swiglu else (data((e, h), 35), data((e, m), 36))
    gx, gh = factors(e, fmt, 3, 0.004), factors(e, fmt, 4, 0.05)
    gw = [factors(e, fmt, 5 + i, 0.002) for i in range(3)]
    counts = torch.tensor(kept, dtype=torch.int32, device="cuda")
    c_dev = torch.tensor([cap], dtype=torch.int32, device="cuda")
    xq, xs = quant(x, fmt, gx, counts, c_dev)
    wq = [(None, None) if t is None else quant(t, fmt, g) for t, g in zip(w, gw)]
    if not swiglu:
        gw[1] = None
    # stale workspace and output
    ws = torch.full((M.moe_expert_ffn_fp4_workspace_size(fmt, act, e, c_max, m, h),), 0x55, dtype=torch.uint8,
                    device="cuda")
    out = torch.full((e, c_max, m), -9.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.moe_expert_ffn_fp4(xq, xs, gx, gh, counts, c_dev, *wq[0], gw[0], b1, *wq[1], gw[1], *wq[2], gw[2], b2, fmt,
                         act, ws, out, st)
    torch.cuda.synchronize()
    status_ok(st)
    nq = e * c_max * h // 2
    hq = ws[:nq].view(e, c_max, h // 2)
    at = (nq + 255) // 256 * 256
    hs = ws[at:at + e * M.moe_fp4_scale_bytes(fmt, c_max, h)].view(e, -1)
    got = out.float().cpu().numpy()
    wv = [None if t[0] is None else values64(*t, fmt, g) for t, g in zip(wq, gw)]
    n, nt = h // BLK[fmt], -(-(h // BLK[fmt]) // 4)
    for j in range(e):
        r = min(kept[j], cap)
        assert (got[j, r:] == -9.0).all() and (hq[j, r:] == 0x55).all()
        if r == 0:
            continue
        one = lambda g: None if g is None else g[j:j + 1]
        xv = values64(xq[j:j + 1, :r], xs[j:j + 1], fmt, one(gx))[0]
        # the hidden: its fp32 value is within tol of the 64-bit one, so its code stands for the
        # rounding of some number within tol; a block's scale may move by one step with it
        pre = xv @ wv[0][j].T
        mag = np.abs(xv) @ np.abs(wv[0][j]).T
        tol = 2.0 ** -23 * (m + 16) * mag + 1e-6 * np.abs(pre)
        if swiglu:
            up = xv @ wv[1][j].T
            tol_up = 2.0 ** -23 * (m + 16) * (np.abs(xv) @ np.abs(wv[1][j]).T) + 1e-6 * np.abs(up)
            sg = 1.0 / (1.0 + np.exp(-pre))
            hid = pre * sg * up
            tol = 1.1 * tol * np.abs(up) + np.abs(pre * sg) * tol_up + 1e-6 * np.abs(hid)
        else:
            b1j = b1[j].float().cpu().numpy().astype(np.float64)
            hid = act64(pre + b1j, act)
            # |act'| <= 1.13; the GELU's own error is below 1e-6 of |x|
            tol = 1.2 * (tol + 2.0 ** -23 * np.abs(b1j)) + 1e-6 * np.abs(pre + b1j)
        tiles = untile(hs[j].cpu().numpy(), r, n)
        assert (tiles[:, n:nt * 4] == 0).all()
        hv = values64(hq[j:j + 1, :r], hs[j:j + 1], fmt, one(gh))[0]
        g = 1.0 if gh is None else float(gh[j])
        sc = tiles[:, :n].astype(np.int64)
        s = np.repeat(np.ldexp(1.0, sc - 127) if fmt == "mx" else E4M3[sc] * g, BLK[fmt], 1)
        amax = np.abs(hid).reshape(r, n, -1).max(2)
        t2 = tol.reshape(r, n, -1).max(2)
        if fmt == "mx":
            lo = np.where(amax - t2 > 0, np.maximum(np.frexp(np.maximum(amax - t2, 1e-300))[1] - 3, -127) + 127, 0)
            hi = np.maximum(np.frexp(np.maximum(amax + t2, 1e-300))[1] - 3, -127) + 127
            assert (((sc >= lo) & (sc <= hi)) | ((amax <= t2) & (sc == 127))).all()
        else:
            lo = nearest(np.clip((amax - t2) / (6 * g) * (1 - 1e-6), 0, 448), E4M3)
            hi = nearest(np.clip((amax + t2) / (6 * g) * (1 + 1e-6), 0, 448), E4M3)
            assert ((sc >= lo) & (sc <= hi)).all()
        # distance to the code's value: half the gap around it, unless saturated or the scale is 0
        live = s > 0
        y = np.where(live, np.abs(hv) / np.where(live, s, 1.0), 0.0)
        k_ = nearest(y, E2M1)
        half_up = np.where(k_ == 7, np.inf, (E2M1[np.minimum(k_ + 1, 7)] - E2M1[k_]) / 2)
        half_dn = (E2M1[k_] - E2M1[np.maximum(k_ - 1, 0)]) / 2
        d = np.where(hv < 0, -1, 1) * hid - np.abs(hv)
        slack = tol + 1e-6 * s
        ok = (d <= half_up * s + slack) & (-d <= np.where(k_ == 0, 0.25 * s, half_dn * s) + slack)
        assert (ok | ~live).all(), j
        # the second product, on the kernel's own hidden
        want = hv @ wv[2][j].T
        mag = np.abs(hv) @ np.abs(wv[2][j]).T
        if b2 is not None:
            want = want + b2[j].float().cpu().numpy()
        assert (np.abs(got[j, :r] - want) <= bound(mag, want, h)).all(), j


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("act", ["relu", "gelu", "swiglu"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_token_spoils_its_own_row_only(fmt, act, bad):
    e, c_max, m, h = 2, 140, 96, 160
    x = data((e, c_max, m), 51)
    w = [quant(data((e, h, m), 52), fmt), quant(data((e, h, m), 53), fmt), quant(data((e, m, h), 54), fmt)]
    if act != "swiglu":
        w[1] = (None, None)
    counts = torch.tensor([c_max, 77], dtype=torch.int32, device="cuda")
    c_dev = torch.tensor([c_max], dtype=torch.int32, device="cuda")
    outs = []
    for spoil in (False, True):
        if spoil:
            x[1, 70, 5] = bad
        q, sc = quant(x, fmt)
        ws = torch.zeros(M.moe_expert_ffn_fp4_workspace_size(fmt, act, e, c_max, m, h), dtype=torch.uint8, device="cuda")
        out = torch.zeros((e, c_max, m), dtype=torch.bfloat16, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        M.moe_expert_ffn_fp4(q, sc, None, None, counts, c_dev, *w[0], None, None, *w[1], None, *w[2], None, None, fmt,
                             act, ws, out, st)
        torch.cuda.synchronize()
        status_ok(st)
        outs.append(out)
    assert torch.isfinite(outs[0].float()).all() and torch.isnan(outs[1][1, 70].float()).all()
    outs[1][1, 70] = outs[0][1, 70]
    assert torch.equal(outs[0], outs[1])


def test_ffn_skips_after_an_error_and_without_rows():
    e, c_max, m, h = 2, 40, 64, 96
    x, w1, w2 = data((e, c_max, m), 1), data((e, h, m), 2), data((e, m, h), 3)
    q = [quant(t, "mx") for t in (x, w1, w2)]
    ws = torch.zeros(M.moe_expert_ffn_fp4_workspace_size("mx", "relu", e, c_max, m, h), dtype=torch.uint8, device="cuda")
    for counts, code in (([0, 0], 0), ([40, 40], M.MOE_ERR_CAPACITY)):
        st = torch.full((1,), code, dtype=torch.int32, device="cuda")
        out = torch.full((e, c_max, m), -9.0, dtype=torch.bfloat16, device="cuda")
        M.moe_expert_ffn_fp4(*q[0], None, None, torch.tensor(counts, dtype=torch.int32, device="cuda"),
                             torch.tensor([c_max], dtype=torch.int32, device="cuda"), *q[1], None, None, None, None,
                             None, *q[2], None, None, "mx", "relu", ws, out, st)
        torch.cuda.synchronize()
        assert int(st.item()) == code and (out == -9.0).all()
