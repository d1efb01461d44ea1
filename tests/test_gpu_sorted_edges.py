"""Sorted rows where the calls can go wrong: idx entries outside the experts."""

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
