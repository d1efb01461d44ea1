"""The gradient of renormalised softmax gates where the forward leaves the normal
numbers: chosen scores that all round to 0, rows with a NaN or +inf."""

import numpy as np
import pytest
import torch

import combine_moe_gate_gb300 as M

from gpu_util import status_ok

pytestmark = pytest.mark.gpu


def forward_then_backward(x, bias, k, dg, scale=1.5):
    s, e = x.shape
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    idx = torch.empty((k, s), dtype=torch.int32, device="cuda")
    gates = torch.empty((k, s), device="cuda")
    d = torch.full((s, e), 7.0, device="cuda")
    M.moe_route_topk(x, bias, k, idx, gates, st, scale=scale, flags=M.MOE_FLAG_NORMALIZE_GATES)
    M.moe_route_bwd(x, idx, dg, d, st, scale=scale, flags=M.MOE_FLAG_NORMALIZE_GATES)
    torch.cuda.synchronize()
    status_ok(st)
    return idx, gates, d


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("e,k,filler", [(24, 3, 0), (60, 4, 30), (256, 8, 200), (1000, 5, 900), (1024, 1, 0)])
def test_gradient_is_zero_where_the_gates_are_the_constant_zero(dt, e, k, filler):
    """A bias picks experts 85 to 125 below the row's maximum: the gates are 0 as
    soon as the chosen scores' sum is, and so is the gradient; above that it is the
    formula's.  `filler` experts at the maximum make the softmax's sum larger."""
    s = 400
    g = torch.Generator().manual_seed(e)
    x = torch.full((s, e), -200.0)
    x[:, e - 1 - filler:] = 3.0                             # the row's maximum, not chosen
    depth = torch.linspace(85.0, 125.0, s)[:, None]
    x[:, :k] = 3.0 - depth - torch.rand((s, k), generator=g) * 2
    bias = torch.zeros(e)
    bias[:k] = 5.0
    x, dg = x.to(dt).cuda(), torch.randn((k, s), generator=g).cuda()
    idx, gates, d = forward_then_backward(x, bias.cuda(), k, dg)
    assert bool((idx < k).all())
    dead = (gates == 0).all(0)
    assert 50 < int(dead.sum()) < 350
    assert bool((d[dead] == 0).all()) and bool((d[:, k:] == 0).all())
    if k == 1:
        assert bool((d == 0).all())
        return
    assert bool((d[~dead][:, :k] != 0).any(1).all())
    x64 = x[:, :k].double().cpu()
    p = torch.softmax(x64, 1)
    dgk = torch.zeros((s, k), dtype=torch.float64).scatter_(1, idx.t().long().cpu(), dg.t().double().cpu())
    want = 1.5 * p * (dgk - (dgk * p).sum(1, keepdim=True))
    # as the 64-bit gradient test derives: differences of terms up to scale |d_gates|, k-term sums
    tol = 1.5 * 2.0 ** -24 * (40 + 4 * k) * dg.abs().max().item()
    live = (~dead).cpu()
    assert bool(((d[:, :k].double().cpu() - want).abs()[live] <= tol).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("e,k", [(7, 2), (60, 4), (256, 8), (1024, 3)])
def test_gradient_shows_a_nan_that_the_gates_show(bad, e, k):
    """A NaN or +inf anywhere in a row makes its gates NaN, the gradient at the
    selection too; other rows and the experts that were not chosen are untouched."""
    s = 50
    g = torch.Generator().manual_seed(k)
    x = torch.randn((s, e), generator=g)
    x[7, e - 1] = x[20, e // 2] = bad
    idx, gates, d = forward_then_backward(x.cuda(), None, k, torch.randn((k, s), generator=g).cuda())
    rows = torch.zeros(s, dtype=torch.bool)
    rows[[7, 20]] = True
    assert np.array_equal(torch.isnan(gates).all(0).cpu().numpy(), rows.numpy())
    chosen = torch.zeros((s, e), dtype=torch.bool).scatter_(1, idx.t().long().cpu(), True)
    assert torch.equal(torch.isnan(d).cpu(), chosen & rows[:, None])
    assert bool((d.cpu()[~chosen] == 0).all())


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_logits_are_aligned_as_a_whole_only(dt):
    """Rows of an odd width are no multiple of 16 bytes; the tensor has to start on 16."""
    s, e, k = 9, 33, 2
    x = torch.randn((s + 1, e), generator=torch.Generator().manual_seed(1)).to(dt).cuda()
    dg = torch.ones((k, s), device="cuda")
    idx, gates, d = forward_then_backward(x[:s], None, k, dg)
    again = forward_then_backward(x[1:].clone(), None, k, dg)   # the same rows, one later
    assert torch.equal(idx[:, 1:], again[0][:, :-1]) and torch.equal(gates[:, 1:], again[1][:, :-1])
    assert torch.equal(d[1:], again[2][:-1])
    before = M.launch_count()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(M.MoEError):
        M.moe_route_topk(x[1:], None, k, idx, gates, st)
    with pytest.raises(M.MoEError):
        M.moe_route_bwd(x[1:], idx, dg, d, st)
    assert M.launch_count() == before


def test_routes_to_masked_experts_take_slots():
    s, e, k = 40, 8, 2
    x = torch.randn((s, e), generator=torch.Generator().manual_seed(2)).cuda()
    x[5:25] = -float("inf")
    idx, gates, _ = forward_then_backward(x, None, k, torch.ones((k, s), device="cuda"))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(M.moe_capacity_workspace_size(s, e, k), dtype=torch.uint8, device="cuda")
    loc, counts = torch.empty_like(idx), torch.empty(e, dtype=torch.int32, device="cuda")
    c_dev = torch.empty(1, dtype=torch.int32, device="cuda")
    M.moe_capacity_locations(idx, e, 0.0, s, ws, loc, counts, c_dev, st)
    torch.cuda.synchronize()
    status_ok(st)
    assert bool((gates[:, 5:25] == 0).all())
    assert torch.equal(counts.long(), idx.long().view(-1).bincount(minlength=e))
    assert int(counts[0]) >= 20 and int(counts[1]) >= 20
