"""Sorted rows where the calls can go wrong: idx entries outside the experts, offsets that do not start at 0, and a
NaN in a live row."""

import pytest
import torch

import combine_moe_gate_gb300 as M
import test_gpu_sorted as S

pytestmark = pytest.mark.gpu


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
