"""Rows sorted by expert on the GPU: the order, the movements and their gradients, the expert
MLP and its gradient, against plain 64-bit forms.

Tolerances are bounds, added up per element: half a step of the output's type (2^-8 of a bf16 value,
2^-24 of an fp32 one) for each rounding, and for a sum of n terms formed in fp32 in any order
n * 2^-24 times the sum of the terms' magnitudes (2 n on the tensor cores, which may cut instead of
round)."""

import pytest
import torch

import combine_moe_gate_gb300 as M

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
U = 2.0 ** -24


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def routes(s, e, k, seed, left_out=0.0, skew=False):
    """Random distinct experts per token [k, s]; a share of routes, and the last token's, without one."""
    g = torch.Generator().manual_seed(seed)
    like = torch.rand((s, e), generator=g)
    if skew:
        like[:, 0] += 1.0
    idx = like.argsort(1, descending=True)[:, :k].t().contiguous().int()
    if left_out:
        idx[torch.rand((k, s), generator=g) < left_out] = -1
        idx[:, -1] = -1
    return idx.cuda()


def plain_order(idx, e):
    """rows, offsets and source, expert by expert."""
    k, s = idx.shape
    flat = idx.flatten().cpu()
    rows, source, offsets = torch.full((k * s,), -1), torch.full((k * s,), -1), [0]
    for j in range(e):
        mine = torch.nonzero(flat == j).flatten()
        rows[mine] = torch.arange(len(mine)) + offsets[-1]
        source[offsets[-1]:offsets[-1] + len(mine)] = mine
        offsets.append(offsets[-1] + len(mine))
    return rows.view(k, s).int().cuda(), torch.tensor(offsets).int().cuda(), source.int().cuda()


def sort(idx, e, st, with_source=True):
    k, s = idx.shape
    rows = torch.full((k, s), -7, dtype=torch.int32, device="cuda")
    offsets = torch.full((e + 1,), -7, dtype=torch.int32, device="cuda")
    source = torch.full((k * s,), -7, dtype=torch.int32, device="cuda") if with_source else None
    ws = torch.full((M.moe_sort_workspace_size(s, e, k),), 0xAB, dtype=torch.uint8, device="cuda")
    M.moe_sort_routes(idx, e, rows, offsets, ws, st, source=source)
    return rows, offsets, source


# one route, a warp's and a CTA's edges, both launch forms, every bucket count's edges
@pytest.mark.parametrize("s,e,k", [(1, 1, 1), (1, 256, 8), (31, 4, 1), (33, 7, 3), (1024, 16, 1), (1025, 256, 1),
                                   (8192, 16, 2), (5461, 60, 3), (16385, 3, 1), (300, 257, 4), (100, 1024, 8),
                                   (40000, 1024, 2), (65536, 64, 2), (70001, 1, 1), (9000, 256, 32)])
@pytest.mark.parametrize("left_out", [0.0, 0.2])
def test_order(s, e, k, left_out):
    idx = routes(s, e, k, s + e, left_out, skew=s % 2 == 1)
    st = status()
    got = sort(idx, e, st)
    for g, want, name in zip(got, plain_order(idx, e), ("rows", "offsets", "source")):
        assert torch.equal(g, want), name
    assert st.item() == 0
    again = sort(idx, e, st, with_source=False)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


@pytest.mark.parametrize("s", [40, 20000])
def test_order_extremes(s):
    st = status()
    idx = torch.full((2, s), -1, dtype=torch.int32, device="cuda")        # no route at all
    rows, offsets, source = sort(idx, 5, st)
    assert (rows == -1).all() and (offsets == 0).all() and (source == -1).all() and st.item() == 0
    idx[:] = 4                                                            # one expert, twice a token
    rows, offsets, source = sort(idx, 5, st)
    assert torch.equal(rows.flatten(), torch.arange(2 * s, device="cuda").int())
    assert offsets.tolist() == [0, 0, 0, 0, 0, 2 * s] and st.item() == 0
    idx[1, s // 2] = 5                                                    # no such expert
    rows, offsets, _ = sort(idx, 5, st)
    assert st.item() == M.MOE_ERR_INVALID_ARG
    before = rows.clone()
    idx[:] = 0
    M.moe_sort_routes(idx, 5, rows, offsets, torch.empty(M.moe_sort_workspace_size(s, 5, 2), dtype=torch.uint8,
                                                         device="cuda"), st)
    assert torch.equal(rows, before)                                      # an error pending: nothing written


def data(shape, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dt)


def near(got, want, bound, name=""):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (name, bad.sum().item(), err.max().item(), (err / bound).nan_to_num().max().item())


MOVES = [(1, 8, 1), (1, 7168, 8), (5, 64, 3), (77, 4096, 2), (300, 520, 4), (33, 2056, 5), (1000, 128, 8), (40, 256, 9),
         (9, 264, 32), (3000, 1024, 6), (257, 16384, 2)]


@pytest.mark.parametrize("s,m,k", MOVES)
@pytest.mark.parametrize("dt", [BF, F32])
def test_movements_and_gradients(s, m, k, dt):
    e = max(k, 8)
    idx = routes(s, e, k, m + s, 0.15 if s > 4 else 0.0)
    rows, offsets, _ = plain_order(idx, e)
    n = s * k + 3
    live, at = rows >= 0, rows.clamp(min=0).long()
    gates = torch.rand((k, s), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) - 0.3
    gates[~live] = float("nan")                        # never used
    x, xs, dy, st = data((s, m), dt, 2), data((n, m), dt, 3), data((s, m), dt, 4), status()
    xs[int(offsets[-1]):] = float("nan")               # no route's rows: never read
    half = HALF[dt]
    gd, xd, xsd, dyd = torch.where(live, gates, 0).double(), x.double(), xs.double(), dy.double()

    # in: a copy, and times the gates, one rounding of the exact product
    for w in (None, gates):
        out = torch.full((n, m), 5.0, dtype=dt, device="cuda")
        M.moe_encode_sorted(x, rows, out, st, gates=w)
        want = torch.full((n, m), 5.0, dtype=torch.float64, device="cuda")
        for r in range(k):
            v = xd if w is None else gd[r, :, None] * xd
            want[at[r][live[r]]] = v[live[r]]
        if w is None:
            assert torch.equal(out.double(), want)
        else:
            near(out, want, half * want.abs(), "in")
        assert (out[int(offsets[-1]):] == 5.0).all()
    # back
    for w in (None, gates):
        y = torch.full((s, m), 5.0, dtype=dt, device="cuda")
        M.moe_decode_sorted(xs, rows, y, st, gates=w)
        want, size = torch.zeros((2, s, m), dtype=torch.float64, device="cuda")
        for r in range(k):
            v = torch.where(live[r, :, None], xsd[at[r]] if w is None else gd[r, :, None] * xsd[at[r]], 0)
            want, size = want + v, size + v.abs()
        near(y, want, half * want.abs() + k * U * size, "back")
        # the gradient of the way in moves rows the same way
        dx = torch.full((s, m), 5.0, dtype=dt, device="cuda")
        M.moe_encode_sorted_bwd(xs, rows, dx, st, gates=w)
        assert torch.equal(dx, y)
    # gradients of the gates
    dots, dsize = torch.zeros((2, k, s), dtype=torch.float64, device="cuda")
    idots, isize = torch.zeros((2, k, s), dtype=torch.float64, device="cuda")
    for r in range(k):
        b = torch.where(live[r, :, None], xsd[at[r]], 0)
        dots[r], dsize[r] = (dyd * b).sum(1), (dyd * b).abs().sum(1)
        idots[r], isize[r] = (xd * b).sum(1), (xd * b).abs().sum(1)
    d_xs, d_gates = torch.full((n, m), 5.0, dtype=dt, device="cuda"), torch.full((k, s), 5.0, device="cuda")
    M.moe_decode_sorted_bwd(dy, xs, rows, gates, d_xs, d_gates, st)
    want = torch.full((n, m), 5.0, dtype=torch.float64, device="cuda")
    for r in range(k):
        want[at[r][live[r]]] = (gd[r, :, None] * dyd)[live[r]]
    near(d_xs, want, half * want.abs(), "d_xs")
    near(d_gates, dots, (m + 8) * U * dsize, "d_gates")
    assert (d_gates[~live] == 0).all()
    dx2, d_in = torch.full((s, m), 5.0, dtype=dt, device="cuda"), torch.full((k, s), 5.0, device="cuda")
    M.moe_encode_sorted_bwd(xs, rows, dx2, st, x=x, gates=gates, d_gates=d_in)
    assert torch.equal(dx2, dx)
    near(d_in, idots, (m + 8) * U * isize, "d_gates in")
    assert st.item() == 0
    first = d_gates.clone()
    M.moe_decode_sorted_bwd(dy, xs, rows, gates, d_xs, d_gates, st)
    assert torch.equal(first, d_gates)                 # the same bits again


def test_gradients_by_differences():
    """Central differences of <dy, way back> in fp32 rows: linear in rows and in gates, so exact but for rounding."""
    s, m, k = 6, 32, 3
    rows, _, _ = plain_order(routes(s, 4, k, 9, 0.2), 4)
    n, st = s * k, status()
    xs, dy, gates = data((n, m), F32, 1), data((s, m), F32, 2), torch.rand((k, s), device="cuda") + 0.5
    d_xs, d_gates = torch.zeros((n, m), device="cuda"), torch.zeros((k, s), device="cuda")
    M.moe_decode_sorted_bwd(dy, xs, rows, gates, d_xs, d_gates, st)

    def value(xs, gates):
        y = torch.empty((s, m), device="cuda")
        M.moe_decode_sorted(xs, rows, y, st, gates=gates)
        return (y.double() * dy.double()).sum()

    for r in range(k):
        for t in range(s):
            lo, hi = gates.clone(), gates.clone()
            lo[r, t] -= 0.5
            hi[r, t] += 0.5
            # y's roundings: k + 1 half steps of values up to 8 in each of m terms, twice
            assert abs((value(xs, hi) - value(xs, lo)).item() - d_gates[r, t].item()) < 2 * m * 4 * 32 * U
    for i in range(0, n, 5):
        lo, hi = xs.clone(), xs.clone()
        lo[i, 3] -= 0.5
        hi[i, 3] += 0.5
        assert abs((value(hi, gates) - value(lo, gates)).item() - d_xs[i, 3].item()) < 2 * 4 * 32 * U


def test_bad_rows_are_reported_and_skipped():
    s, m, k, n = 40, 64, 2, 80
    rows = torch.arange(80, device="cuda").int().view(k, s)
    rows[0, 7], rows[1, 9] = n, -2
    x, st = data((s, m), BF, 1), status()
    out = torch.zeros((n, m), dtype=BF, device="cuda")
    M.moe_encode_sorted(x, rows, out, st)
    assert st.item() == M.MOE_ERR_INVALID_ARG
    assert (out[7] == 0).all() and (out[49] == 0).all()
    st = status()
    y = torch.zeros((s, m), dtype=BF, device="cuda")
    M.moe_decode_sorted(out, rows, y, st)
    assert st.item() == M.MOE_ERR_INVALID_ARG


# ------------------------------------------------------------- the expert MLP
def act64(a, b, act):
    if act == "relu":
        return torch.relu(a)
    return torch.nn.functional.gelu(a) if act == "gelu" else torch.nn.functional.silu(a) * b


def experts(counts, m, h, act, seed=0, extra=5):
    """Inputs of an MLP over the given rows per expert, NaN in the rows of no expert."""
    e, total = len(counts), sum(counts)
    n = total + extra
    off = torch.tensor([0] + counts).cumsum(0).int().cuda()
    p = {"x": data((n, m), BF, seed), "w1": data((e, h, m), BF, seed + 1) * m ** -0.5,
         "w3": data((e, h, m), BF, seed + 2) * m ** -0.5 if act == "swiglu" else None,
         "w2": data((e, m, h), BF, seed + 3) * h ** -0.5, "off": off, "n": n, "total": total,
         "b1": None if act == "swiglu" else data((e, h), BF, seed + 4),
         "b2": None if act == "swiglu" else data((e, m), BF, seed + 5), "d_out": data((n, m), BF, seed + 6)}
    p["x"][total:] = float("nan")
    p["d_out"][total:] = float("nan")
    return p


def forward(p, act, train=True):
    n, m = p["x"].shape
    h = p["w1"].shape[1]
    st = status()
    hid, out = torch.full((n, h), 5.0, dtype=BF, device="cuda"), torch.full((n, m), 5.0, dtype=BF, device="cuda")
    pre = torch.full((n, 2 * h if act == "swiglu" else h), 5.0, dtype=BF, device="cuda") if train else None
    M.moe_expert_ffn_sorted(p["x"], p["off"], p["w1"], p["b1"], p["w3"], p["w2"], p["b2"], act, hid, out, st, pre=pre)
    assert st.item() == 0
    return hid, pre, out


SHAPES = [([1], 8, 8), ([33], 520, 24), ([64], 264, 40), ([2, 0, 40, 11], 1032, 88), ([50, 15], 264, 40), ([3, 0, 1], 64, 40), ([0, 0, 65], 72, 136), ([64, 128, 256, 1, 0, 255, 257], 128, 256),
          ([500, 2, 700], 264, 520), ([0, 33, 31, 32, 97], 1024, 704), ([1] * 40 + [0] * 20, 256, 96),
          ([1300, 0, 300, 64], 520, 1040)]


@pytest.mark.parametrize("counts,m,h", SHAPES)
@pytest.mark.parametrize("act", ["relu", "gelu", "swiglu"])
def test_mlp_and_gradient(counts, m, h, act):
    p = experts(counts, m, h, act)
    hid, pre, out = forward(p, act)
    T = p["total"]
    for t in (hid, pre, out):
        assert (t[T:] == 5.0).all()                     # rows of no expert: not written
    plain_hid, _, plain_out = forward(p, act, train=False)
    assert torch.equal(plain_hid, hid) and torch.equal(plain_out, out)
    swiglu, half = act == "swiglu", HALF[BF]
    e = len(counts)
    gdt = [BF, F32]
    grads = []
    for dt in gdt:
        g = {"d_x": torch.full_like(p["x"], 5.0)}
        for name in ("w1", "w3", "w2", "b1", "b2"):
            if p[name] is not None:
                g["d_" + name] = torch.full(p[name].shape, 5.0, dtype=dt, device="cuda")
        ws = torch.full((M.moe_expert_ffn_sorted_bwd_workspace_size(act, e, p["n"], m, h),), 0xFF, dtype=torch.uint8,
                        device="cuda")                  # NaN patterns
        st = status()
        pre[T:] = hid[T:] = float("nan")
        M.moe_expert_ffn_sorted_bwd(p["x"], hid, pre, p["off"], p["w1"], p["w3"], p["w2"], act, p["d_out"], ws,
                                    g["d_x"], g["d_w1"], g.get("d_w3"), g["d_w2"], g.get("d_b1"), g.get("d_b2"), st)
        assert st.item() == 0 and (g["d_x"][T:] == 5.0).all()
        grads.append(g)
    assert torch.equal(grads[0]["d_x"][:T], grads[1]["d_x"][:T])
    lo = 0
    for j, c in enumerate(counts):
        r = slice(lo, lo + c)
        lo += c
        if c == 0:
            for g in grads:
                for name in g:
                    if name != "d_x":
                        assert (g[name][j] == 0).all(), name
            continue
        x, w1, w2 = p["x"][r].double(), p["w1"][j].double(), p["w2"][j].double()
        w3 = p["w3"][j].double() if swiglu else None
        a = x @ w1.t() + (0 if swiglu else p["b1"][j].double())
        b = x @ w3.t() if swiglu else None
        ea = 2 * (m + 1) * U * (x.abs() @ w1.abs().t() + (0 if swiglu else p["b1"][j].double().abs()))
        got_pre = pre[r].double()
        near(got_pre[:, :h], a, half * a.abs() * 1.01 + ea, "pre")
        want = act64(a, b, act)
        if swiglu:
            eb = 2 * m * U * (x.abs() @ w3.abs().t())
            near(got_pre[:, h:], b, half * b.abs() * 1.01 + eb, "pre b")
            eh = 1.1 * ea * b.abs() + torch.nn.functional.silu(a).abs() * eb + 8 * U * want.abs()
        else:
            eh = 1.13 * ea + 6e-7                       # |act'| and the GELU's approximation
        near(hid[r], want, half * want.abs() * 1.01 + eh, "hid")
        hd = hid[r].double()                            # the second product reads the stored hidden
        o = hd @ w2.t() + (0 if swiglu else p["b2"][j].double())
        eo = 2 * (h + 1) * U * (hd.abs() @ w2.abs().t() + (0 if swiglu else p["b2"][j].double().abs()))
        near(out[r], o, half * o.abs() * 1.01 + eo, "out")

        # the gradient, from the stored hid and pre
        do = p["d_out"][r].double()
        pr = got_pre.clone().requires_grad_(True)
        hh = act64(pr[:, :h], pr[:, h:], act)
        dh = do @ w2
        (dp,) = torch.autograd.grad(hh, pr, dh)
        edh = 2 * m * U * (do.abs() @ w2.abs())
        # d_pre: the product's sums, the derivative's evaluation (1e-6 of it, and of d_hid), one rounding
        slope = torch.autograd.grad(act64(pr[:, :h], pr[:, h:], act), pr, torch.ones_like(dh))[0].abs()
        two = torch.cat((edh, edh), 1) if swiglu else edh
        dh2 = torch.cat((dh, dh), 1) if swiglu else dh
        scale2 = torch.cat((got_pre[:, h:].abs(), got_pre[:, :h].abs()), 1) if swiglu else 1.0
        ep = half * dp.abs() * 1.01 + slope * two + 2e-6 * dh2.abs() * (scale2 + slope)
        wcat = torch.cat((w1, w3)) if swiglu else w1
        dx = dp @ wcat
        H = wcat.shape[0]
        near(grads[0]["d_x"][r], dx, half * dx.abs() * 1.01 + ep @ wcat.abs() * 1.01 + 2 * H * U * (dp.abs() @ wcat.abs()),
             "d_x")
        for g, gh in zip(grads, (half, U)):
            dw = dp.t() @ x
            bound = ep.t() @ x.abs() * 1.01 + 2 * c * U * (dp.abs().t() @ x.abs())
            near(g["d_w1"][j], dw[:h], gh * dw[:h].abs() * 1.01 + bound[:h], "d_w1")
            if swiglu:
                near(g["d_w3"][j], dw[h:], gh * dw[h:].abs() * 1.01 + bound[h:], "d_w3")
            else:
                near(g["d_b1"][j], dp.sum(0), gh * dp.sum(0).abs() * 1.01 + ep.sum(0) + 2 * c * U * dp.abs().sum(0), "d_b1")
                near(g["d_b2"][j], do.sum(0), gh * do.sum(0).abs() * 1.01 + 2 * c * U * do.abs().sum(0), "d_b2")
            dw2 = do.t() @ hd
            near(g["d_w2"][j], dw2, gh * dw2.abs() * 1.01 + 2 * c * U * (do.abs().t() @ hd.abs()), "d_w2")


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_mlp_is_the_buffer_form_row_for_row(act):
    """The same rows through moe_expert_ffn's [e, c_max, m] buffer: the same bits."""
    counts, m, h = [70, 0, 300, 129], 256, 320
    p = experts(counts, m, h, act)
    hid, _, out = forward(p, act)
    c = max(counts)
    buf = torch.zeros((4, c, m), dtype=BF, device="cuda")
    lo = 0
    for j, q in enumerate(counts):
        buf[j, :q] = p["x"][lo:lo + q]
        lo += q
    cnt, c_dev, st = torch.tensor(counts).int().cuda(), torch.tensor([c]).int().cuda(), status()
    ws = torch.empty(M.moe_expert_ffn_workspace_size(M.MOE_BF16, act, 4, c, m, h), dtype=torch.uint8, device="cuda")
    ref = torch.zeros((4, c, m), dtype=BF, device="cuda")
    M.moe_expert_ffn(buf, cnt, c_dev, p["w1"], p["b1"], p["w3"], p["w2"], p["b2"], act, ws, ref, st)
    lo = 0
    for j, q in enumerate(counts):
        assert torch.equal(out[lo:lo + q], ref[j, :q])
        lo += q


@pytest.mark.parametrize("bad", ["descending", "beyond", "negative"])
def test_bad_offsets_are_reported(bad):
    p = experts([10, 20, 30], 64, 64, "gelu")
    p["off"][1 if bad == "descending" else 3 if bad == "beyond" else 0] = {"descending": 50, "beyond": 10 ** 6,
                                                                         "negative": -4}[bad]
    n, st = p["n"], status()
    hid, out = torch.zeros((n, 64), dtype=BF, device="cuda"), torch.zeros((n, 64), dtype=BF, device="cuda")
    M.moe_expert_ffn_sorted(p["x"], p["off"], p["w1"], p["b1"], None, p["w2"], p["b2"], "gelu", hid, out, st)
    assert st.item() == M.MOE_ERR_INVALID_ARG


def test_no_rows_at_all():
    p = experts([0, 0, 0], 64, 64, "gelu", extra=9)
    hid, pre, out = forward(p, "gelu")
    assert (out == 5.0).all() and (hid == 5.0).all()
