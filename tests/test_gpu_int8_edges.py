"""8-bit integer experts where the calls can go wrong: offsets that do not start at 0."""

import pytest
import torch

import combine_moe_gate_gb300 as M
import test_gpu_int8 as S

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("n", [2, 6, 90])
def test_offsets_that_do_not_start_at_0_are_reported(n):
    a, w, st = S.codes((n, 64), 1), S.codes((4, 64, 64), 2), S.status()
    off = torch.tensor([1, 1, 2, 2, n]).int().cuda()
    one, sw = torch.ones(n, device="cuda"), torch.ones((4, 64), device="cuda")
    ws = torch.empty(M.moe_product_int8_workspace_size(4, n, 64, 64), dtype=torch.uint8, device="cuda")
    M.moe_product_int8(a, one, off, w, sw, None, ws, torch.zeros((n, 64), device="cuda"), st)
    assert st.item() == M.MOE_ERR_INVALID_ARG
    st = S.status()
    ws = torch.zeros(M.moe_expert_ffn_int8_workspace_size("gelu", 4, n, 64, 64), dtype=torch.uint8, device="cuda")
    M.moe_expert_ffn_int8(a, one, off, w, sw, None, None, None, w, sw, None, "gelu", ws,
                          torch.zeros((n, 64), dtype=BF, device="cuda"), st)
    assert st.item() == M.MOE_ERR_INVALID_ARG
