"""8-bit integer rows on the GPU: the quantiser, the grouped product and the expert MLP, against
64-bit forms.

Codes and scales have to be equal: the definition fixes every fp32 step.  Products: the integer sum is
exact (k <= 1024), else an fp32 sum of k products, which may cut instead of round (2 k * 2^-24
of the magnitudes' sum); the scales' product, its product with the sum, and the output are rounded
once each (2^-24 of the value; half a step of the output's type)."""

import pytest
import torch

import combine_moe_gate_gb300 as M

pytestmark = pytest.mark.gpu

BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
U = 2.0 ** -24


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def plain_quantize(x):
    """The definition with fp32 steps (torch divides tensors, multiplies and rounds as IEEE does; by a
    Python number it would multiply with the reciprocal)."""
    x = x.float()
    bad = ~torch.isfinite(x).all(-1)
    amax = torch.where(bad, 1.0, x.abs().nan_to_num(posinf=0.0).amax(-1))
    live = amax >= 2.0 ** -100
    top = torch.full_like(amax, 127.0)
    scale = torch.where(bad, torch.nan, torch.where(live, amax / top, 1.0))
    inv = torch.where(live, top / amax, 0.0)
    q = torch.where(bad[..., None], 0.0, (x * inv[..., None]).round())
    return q.to(I8), scale


def same(a, b):
    return torch.equal(a.view(torch.int32), b.view(torch.int32)) or (
        torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num()))


# one warp's row and its edges, the register forms' limits, a row read twice, one row and many
@pytest.mark.parametrize("s,cols", [(1, 16), (1, 7168), (5, 2048), (3, 2064), (700, 48), (33, 4096), (9, 8208), (2, 16384),
                                    (3, 20480), (5000, 256)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_quantise(s, cols, dt):
    x = torch.randn((s, cols), generator=gen(s), device="cuda").mul_(3.0)
    x *= torch.exp(torch.randn((s, 1), generator=gen(1), device="cuda") * 8)
    x[s // 2, cols // 3] = -50.0
    x = x.to(dt)
    q, scale, st = torch.full((s, cols), 77, dtype=I8, device="cuda"), torch.full((s,), 9.0, device="cuda"), status()
    M.moe_quantize_rows_int8(x, q, scale, st)
    wq, ws = plain_quantize(x)
    assert torch.equal(q, wq) and same(scale, ws) and st.item() == 0
    # into sorted rows: every route's row a copy, the others untouched
    k, n = 3, 3 * s + 4
    rows = torch.randperm(n, generator=torch.Generator().manual_seed(2))[: k * s].view(k, s).int()
    rows[torch.rand((k, s), generator=torch.Generator().manual_seed(3)) < 0.3] = -1
    rows = rows.cuda()
    fq, fs = torch.full((n, cols), 77, dtype=I8, device="cuda"), torch.full((n,), 9.0, device="cuda")
    M.moe_quantize_rows_int8(x, fq, fs, st, rows=rows)
    want_q, want_s = torch.full_like(fq, 77), torch.full_like(fs, 9.0)
    for r in range(k):
        live = rows[r] >= 0
        want_q[rows[r][live].long()] = wq[live]
        want_s[rows[r][live].long()] = ws[live]
    assert torch.equal(fq, want_q) and same(fs, want_s) and st.item() == 0


def test_quantise_edges():
    x = torch.zeros((8, 64), device="cuda")
    x[1, 5] = float("nan")
    x[2, 6] = float("inf")
    x[3, :] = 2.0 ** -101
    x[4, 0], x[4, 1] = 2.0 ** -100, -(2.0 ** -100)
    x[5, :3] = torch.tensor([3.0e38, -3.0e38, 1.0e36])
    x[6, 0], x[6, 1:] = 127.0, torch.arange(63, device="cuda") + 0.5      # ties to even
    q, scale, st = torch.empty((8, 64), dtype=I8, device="cuda"), torch.empty(8, device="cuda"), status()
    M.moe_quantize_rows_int8(x, q, scale, st)
    wq, ws = plain_quantize(x)
    assert torch.equal(q, wq) and same(scale, ws)
    assert scale[0] == 1 and scale[3] == 1 and scale[1].isnan() and scale[2].isnan()
    assert q[6, 1:5].tolist() == [0, 2, 2, 4] and q[4, :2].tolist() == [127, -127]


def test_quantise_reports_bad_rows():
    x, st = torch.ones((4, 32), device="cuda"), status()
    q, scale = torch.zeros((6, 32), dtype=I8, device="cuda"), torch.zeros(6, device="cuda")
    M.moe_quantize_rows_int8(x, q, scale, st, rows=torch.tensor([[0, 6, -1, 3]], dtype=torch.int32, device="cuda"))
    assert st.item() == M.MOE_ERR_INVALID_ARG


def codes(shape, seed, lo=-127, hi=128):
    return torch.randint(lo, hi, shape, dtype=I8, generator=gen(seed), device="cuda")


def offsets(counts):
    return torch.tensor([0] + list(counts)).cumsum(0).int().cuda()


def near(got, want, bound, name=""):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (name, bad.sum().item(), err.max().item(), (err / bound).nan_to_num().max().item())


def product(a, sa, off, w, sw, bias, dt):
    n, e, no = a.shape[0], w.shape[0], w.shape[1]
    ws = torch.full((M.moe_product_int8_workspace_size(e, n, a.shape[1], no),), 0xFF, dtype=torch.uint8, device="cuda")
    out, st = torch.full((n, no), 5.0, dtype=dt, device="cuda"), status()
    M.moe_product_int8(a, sa, off, w, sw, bias, ws, out, st)
    assert st.item() == 0
    return out


# few rows (one launch of dot products) and many; K and widths inside a tile and over several; uneven cuts
PRODUCTS = [([1], 16, 8), ([20], 4112, 24), ([64], 4096, 136), ([3, 0, 40, 21], 2064, 40), ([65], 4112, 24), ([1], 4096, 520), ([2, 0, 1], 48, 24), ([0, 5, 0, 3], 272, 264), ([8], 1040, 40), ([9], 16, 8), ([70], 16, 8),
            ([0, 31, 1, 0, 64], 128, 256), ([33, 193, 0, 385], 144, 136), ([192, 191, 1], 64, 512), ([961], 1024, 128),
            ([7] * 60, 256, 72), ([500, 0, 1300], 2064, 776), ([40, 3], 8192, 1032)]


@pytest.mark.parametrize("counts,k,n_out", PRODUCTS)
@pytest.mark.parametrize("dt", [BF, F32])
def test_product(counts, k, n_out, dt):
    e, total = len(counts), sum(counts)
    n = total + (0 if total <= 8 else 5)
    a, w = codes((n, k), 1), codes((e, n_out, k), 2)
    sa, sw = torch.rand(n, generator=gen(3), device="cuda") + 0.1, torch.rand((e, n_out), generator=gen(4), device="cuda")
    sa[total:] = float("nan")
    bias = torch.randn((e, n_out), generator=gen(5), device="cuda").bfloat16() * 100 if dt is BF else None
    out = product(a, sa, offsets(counts), w, sw, bias, dt)
    assert (out[total:] == 5.0).all()
    lo, half = 0, HALF[dt]
    for j, c in enumerate(counts):
        r = slice(lo, lo + c)
        lo += c
        ad, wd, s2 = a[r].double(), w[j].double(), sa[r, None].double() * sw[j].double()
        acc = ad @ wd.t()
        want = acc * s2 + (bias[j].double() if bias is not None else 0)
        fsum = 0.0 if k <= 1024 else 2 * k * U * (ad.abs() @ wd.abs().t()) * s2
        near(out[r], want, half * want.abs() * 1.01 + 3 * U * (acc * s2).abs() + fsum)
    assert torch.equal(out[:total], product(a, sa, offsets(counts), w, sw, bias, dt)[:total])


@pytest.mark.parametrize("n", [3, 40, 90])
def test_product_largest_codes_are_exact(n):
    """All codes -128 (k 1024: the sum is 2^24) and alternating ends: integers come out exactly."""
    k = 1024
    a, w = torch.full((n, k), -128, dtype=I8, device="cuda"), torch.full((1, 16, k), -128, dtype=I8, device="cuda")
    w[0, 1], w[0, 2, ::2], w[0, 3] = 127, 127, 0
    one = torch.ones(n, device="cuda")
    out = product(a, one, None, w, torch.ones((1, 16), device="cuda"), None, F32)
    assert torch.equal(out.double(), a.double() @ w[0].double().t())


def test_product_position_of_every_code():
    """One non-zero code a row and a channel: the sum picks it out (an order mistake in K shows)."""
    k = 256
    a = torch.zeros((k, k), dtype=I8, device="cuda")
    a[torch.arange(k), torch.arange(k)] = 1
    w = codes((1, 264, k), 7, -128)
    out = product(a, torch.ones(k, device="cuda"), None, w, torch.ones((1, 264), device="cuda"), None, F32)
    assert torch.equal(out, w[0].t().float())
    out = product(a[5:11].contiguous(), torch.ones(6, device="cuda"), None, w, torch.ones((1, 264), device="cuda"), None, F32)
    assert torch.equal(out, w[0].t()[5:11].float())


@pytest.mark.parametrize("rows,experts", [(2, 96), (33, 64), (64, 48), (100, 48), (128, 40), (150, 40), (192, 40), (500, 12)])
def test_product_of_many_tiles_a_pair(rows, experts):
    """Several tiles of many stages for each pair of multiprocessors, in every layout of tensor memory; fp32
    sums of small codes are exact, so the result is."""
    k, n_out = 1920, 2056
    n = rows * experts
    a, w = codes((n, k), 1, -15, 16), codes((experts, n_out, k), 2, -15, 16)     # sums below 2^19
    sa, sw = torch.full((n,), 0.5, device="cuda"), torch.full((experts, n_out), 0.25, device="cuda")
    out = product(a, sa, offsets([rows] * experts), w, sw, None, F32)
    for j in range(experts):
        want = (a[j * rows:(j + 1) * rows].float() @ w[j].float().t()) * 0.125
        assert torch.equal(out[j * rows:(j + 1) * rows], want), j


def test_product_nan_scale_stays_in_its_row():
    a, w = codes((50, 64), 1), codes((1, 64, 64), 2)
    sa = torch.ones(50, device="cuda")
    sa[7] = float("nan")
    out = product(a, sa, None, w, torch.ones((1, 64), device="cuda"), None, BF)
    assert out[7].isnan().all() and not out[:7].isnan().any() and not out[8:].isnan().any()


@pytest.mark.parametrize("n", [6, 90])
@pytest.mark.parametrize("bad", [[0, 40, 3], [0, 2, 10 ** 6], [-1, 2, 4]])
def test_bad_offsets_are_reported(n, bad):
    a, w, st = codes((n, 64), 1), codes((2, 64, 64), 2), status()
    ws = torch.empty(M.moe_product_int8_workspace_size(2, n, 64, 64), dtype=torch.uint8, device="cuda")
    out = torch.zeros((n, 64), device="cuda")
    M.moe_product_int8(a, torch.ones(n, device="cuda"), torch.tensor(bad).int().cuda(), w,
                       torch.ones((2, 64), device="cuda"), None, ws, out, st)
    assert st.item() == M.MOE_ERR_INVALID_ARG


FFNS = [([1], 16, 16), ([40, 0, 24], 1056, 80), ([50, 15], 1056, 80), ([1, 0, 2], 64, 48), ([0, 8], 1024, 272), ([9, 0, 33], 128, 112), ([200, 0, 1, 64, 390], 256, 528),
        ([3] * 50 + [0] * 14, 512, 192), ([700, 300], 1040, 2080)]


@pytest.mark.parametrize("counts,m,h", FFNS)
@pytest.mark.parametrize("act", ["relu", "gelu", "swiglu"])
def test_mlp(counts, m, h, act):
    e, total, swiglu = len(counts), sum(counts), act == "swiglu"
    n = total + (0 if total <= 8 else 7)
    x, sx = codes((n, m), 1), torch.rand(n, generator=gen(2), device="cuda") * 0.02 + 0.01
    sx[total:] = float("nan")

    def weight(rows, cols, seed):
        return codes((e, rows, cols), seed), (torch.rand((e, rows), generator=gen(seed + 1), device="cuda") + 0.5) / 73 * cols ** -0.5

    w1, s1 = weight(h, m, 3)
    w3, s3 = weight(h, m, 5) if swiglu else (None, None)
    w2, s2 = weight(m, h, 7)
    b1 = None if swiglu else torch.randn((e, h), generator=gen(9), device="cuda").bfloat16()
    b2 = None if swiglu else torch.randn((e, m), generator=gen(10), device="cuda").bfloat16()
    ws = torch.full((M.moe_expert_ffn_int8_workspace_size(act, e, n, m, h),), 0xFF, dtype=torch.uint8, device="cuda")
    out, st = torch.full((n, m), 5.0, dtype=BF, device="cuda"), status()
    M.moe_expert_ffn_int8(x, sx, offsets(counts), w1, s1, b1, w3, s3, w2, s2, b2, act, ws, out, st)
    assert st.item() == 0 and (out[total:] == 5.0).all()
    hid = ws[: n * h * 2].view(BF).view(n, h)
    at = (n * h * 2 + 255) // 256 * 256
    hs = ws[at: at + 4 * n].view(F32)
    hq, want_hs = plain_quantize(hid[:total])
    assert torch.equal(hs[:total], want_hs)
    lo, half = 0, HALF[BF]
    for j, c in enumerate(counts):
        r = slice(lo, lo + c)
        lo += c
        xd, s = x[r].double(), sx[r, None].double()
        fsum = 0.0 if m <= 1024 else 2 * m * U

        def up(w, sw):
            sc = s * sw[j].double()
            v = xd @ w[j].double().t() * sc
            return v, 3 * U * v.abs() + fsum * (xd.abs() @ w[j].double().abs().t()) * sc

        a, ea = up(w1, s1)
        if swiglu:
            b, eb = up(w3, s3)
            want = torch.nn.functional.silu(a) * b
            eh = 1.1 * ea * b.abs() + torch.nn.functional.silu(a).abs() * eb + 8 * U * want.abs()
        else:
            a = a + b1[j].double()
            ea = ea + U * a.abs()
            want = torch.relu(a) if act == "relu" else torch.nn.functional.gelu(a)
            eh = 1.13 * ea + 6e-7
        near(hid[r], want, half * want.abs() * 1.01 + eh, "hid")
        hd, s = hq[r].double(), want_hs[r, None].double() * s2[j].double()
        acc = hd @ w2[j].double().t()
        o = acc * s + (0 if swiglu else b2[j].double())
        fs = 0.0 if h <= 1024 else 2 * h * U * (hd.abs() @ w2[j].double().abs().t()) * s
        near(out[r], o, half * o.abs() * 1.01 + 3 * U * (acc * s).abs() + fs, "out")


def test_mlp_of_one_expert_without_offsets():
    for n in (4, 30, 100):
        x, sx = codes((n, 64), 1), torch.full((n,), 0.01, device="cuda")
        w1, w2 = codes((1, 96, 64), 2), codes((1, 64, 96), 3)
        s1, s2 = torch.full((1, 96), 0.01, device="cuda"), torch.full((1, 64), 0.01, device="cuda")
        outs = []
        for off in (None, offsets([n])):
            ws = torch.empty(M.moe_expert_ffn_int8_workspace_size("gelu", 1, n, 64, 96), dtype=torch.uint8, device="cuda")
            out, st = torch.zeros((n, 64), dtype=BF, device="cuda"), status()
            M.moe_expert_ffn_int8(x, sx, off, w1, s1, None, None, None, w2, s2, None, "gelu", ws, out, st)
            assert st.item() == 0
            outs.append(out)
        assert torch.equal(*outs) and outs[0].abs().sum() > 0


def test_a_stalled_product_reports_and_the_next_call_is_unharmed():
    a, w = codes((300, 256), 1), codes((2, 264, 256), 2)
    sa, sw, off = torch.rand(300, device="cuda"), torch.rand((2, 264), device="cuda"), offsets([100, 200])
    first = product(a, sa, off, w, sw, None, BF)
    ws = torch.empty(M.moe_product_int8_workspace_size(2, 300, 256, 264), dtype=torch.uint8, device="cuda")
    out, st = torch.zeros((300, 264), dtype=BF, device="cuda"), status()
    M.moe_debug_stall_gemms(1)
    try:
        M.moe_product_int8(a, sa, off, w, sw, None, ws, out, st)
        assert st.item() == M.MOE_ERR_TIMEOUT
    finally:
        M.moe_debug_stall_gemms(0)
    assert torch.equal(product(a, sa, off, w, sw, None, BF), first)
