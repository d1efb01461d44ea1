"""Sorted rows where the calls can go wrong: idx entries outside the experts, offsets that do not start at 0, a
NaN in a live row, and the gradient over several tiles a pair of multiprocessors."""

import pytest
import torch

import combine_moe_gate_gb300 as M
import test_gpu_sorted as S

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


# one launch; counted and placed from registers; placed in two passes (more than 524288 routes)
@pytest.mark.parametrize("s", [40, 20000, 300000])
@pytest.mark.parametrize("entry", [-2 ** 31, -2 ** 31 + 1, -2, 5, 2 ** 31 - 1])
def test_order_reports_any_entry_outside_the_experts(s, entry):
    for r, t in ((0, 0), (1, s // 2), (1, s - 1)):
        idx = torch.randint(0, 5, (2, s), generator=torch.Generator().manual_seed(s)).int().cuda()
        idx[r, t] = entry
        st = S.status()
        S.sort(idx, 5, st)
        assert st.item() == M.MOE_ERR_INVALID_ARG, (r, t)
    idx[r, t] = -1                                        # a route without an expert is none of them
    st = S.status()
    rows, offsets, source = S.sort(idx, 5, st)
    assert st.item() == 0 and rows[r, t].item() == -1 and source[-1].item() == -1


# few rows (dot products) and many (tiles)
@pytest.mark.parametrize("counts", [[10, 5, 3], [100, 20, 30]])
@pytest.mark.parametrize("act", ["relu", "gelu", "swiglu"])
def test_offsets_that_do_not_start_at_0_are_reported(counts, act):
    p = S.experts(counts, 64, 64, act)
    hid, pre, out = S.forward(p, act)
    p["off"][0] = 3
    n, st = p["n"], S.status()
    M.moe_expert_ffn_sorted(p["x"], p["off"], p["w1"], p["b1"], p["w3"], p["w2"], p["b2"], act, torch.zeros_like(hid),
                            torch.zeros_like(out), st)
    assert st.item() == M.MOE_ERR_INVALID_ARG
    st = S.status()
    ws = torch.zeros(M.moe_expert_ffn_sorted_bwd_workspace_size(act, 3, n, 64, 64), dtype=torch.uint8, device="cuda")
    g = {k: torch.zeros_like(p[k]) for k in ("x", "w1", "w2")}
    M.moe_expert_ffn_sorted_bwd(p["x"], hid, pre, p["off"], p["w1"], p["w3"], p["w2"], act, p["d_out"], ws, g["x"], g["w1"],
                                torch.zeros_like(p["w1"]) if act == "swiglu" else None, g["w2"], None, None, st)
    assert st.item() == M.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("counts", [[5, 9, 2], [40, 0, 300]])
@pytest.mark.parametrize("act", ["relu", "gelu", "swiglu"])
@pytest.mark.parametrize("train", [False, True])
def test_a_nan_stays_in_its_row(counts, act, train):
    p = S.experts(counts, 72, 136, act)
    T, at = p["total"], 7
    p["x"][at, 3] = float("nan")
    hid, pre, out = S.forward(p, act, train=train)
    for t in (hid, out) + ((pre,) if train else ()):
        assert t[at].isnan().all()
        assert not t[:at].isnan().any() and not t[at + 1:T].isnan().any()


# 64 uneven experts, some without rows: 288 derivative tiles of 256 x 256 and more, ragged in rows and in columns,
# with tiles whose last columns only half of the warps have (h = 776) and K blocks inside and past one (m)
UNEVEN = [0, 1, 33, 129, 257, 300, 64, 65] * 8


@pytest.mark.parametrize("m,h", [(64, 776), (264, 832)])
@pytest.mark.parametrize("act", ["swiglu", "gelu"])
def test_gradient_over_several_tiles_a_pair(m, h, act):
    S.test_mlp_and_gradient(UNEVEN, m, h, act)          # against 64 bits


@pytest.mark.parametrize("m,h", [(64, 776), (128, 832)])
@pytest.mark.parametrize("act", ["swiglu", "gelu"])
def test_gradient_of_many_tiles_is_the_buffer_forms(m, h, act):
    """The same rows through the [e, c_max, m] buffer's gradient, and twice: the same bits."""
    p = S.experts(UNEVEN, m, h, act)
    e, n, T, c, swiglu = len(UNEVEN), p["n"], p["total"], max(UNEVEN), act == "swiglu"
    hid, pre, out = S.forward(p, act)

    def grads():
        g = {k: torch.full_like(p[k], 5.0) for k in ("w1", "w3", "w2", "b1", "b2") if p[k] is not None}
        return g, (g["w1"], g.get("w3"), g["w2"], g.get("b1"), g.get("b2"))

    runs = []
    for _ in range(2):
        g, args = grads()
        d_x, st = torch.full_like(p["x"], 5.0), S.status()
        ws = torch.full((M.moe_expert_ffn_sorted_bwd_workspace_size(act, e, n, m, h),), 0xFF, dtype=torch.uint8, device="cuda")
        M.moe_expert_ffn_sorted_bwd(p["x"], hid, pre, p["off"], p["w1"], p["w3"], p["w2"], act, p["d_out"], ws, d_x, *args, st)
        assert st.item() == 0
        runs.append((g, d_x[:T].clone()))
    assert torch.equal(runs[0][1], runs[1][1]) and all(torch.equal(runs[0][0][k], runs[1][0][k]) for k in runs[0][0])

    def buffer(rows):
        b = torch.zeros((e, c, rows.shape[1]), dtype=BF, device="cuda")
        lo = 0
        for j, q in enumerate(UNEVEN):
            b[j, :q] = rows[lo:lo + q]
            lo += q
        return b

    g, args = grads()
    cnt, c_dev, st = torch.tensor(UNEVEN).int().cuda(), torch.tensor([c]).int().cuda(), S.status()
    ws = torch.zeros(M.moe_expert_ffn_bwd_workspace_size(M.MOE_BF16, act, e, c, m, h), dtype=torch.uint8, device="cuda")
    d_buf = torch.zeros((e, c, m), dtype=BF, device="cuda")
    M.moe_expert_ffn_bwd_saved(buffer(p["x"]), buffer(hid), buffer(pre), cnt, c_dev, p["w1"], p["w3"], p["w2"], act,
                               buffer(p["d_out"]), ws, d_buf, *args, st)
    assert st.item() == 0
    assert all(torch.equal(g[k], runs[0][0][k]) for k in g)
    lo = 0
    for j, q in enumerate(UNEVEN):
        assert torch.equal(d_buf[j, :q], runs[0][1][lo:lo + q]), j
        lo += q
