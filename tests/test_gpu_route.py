"""moe_route_topk and moe_route_bwd on the GPU against plain 64-bit forms.

Tolerances, derived from fp32: a score carries the rounding of its exponent's
argument (softmax: |l - max| <= 32 units of 2^-24 relative) and a few units
from exp, the sum and the division, so 6e-6 relative covers a gate; choices
(scores below 1, a bias below 1, a sum of two) are off by less than 2e-6, so a
token whose 64-bit margins all exceed that must route exactly alike."""

import numpy as np
import pytest
import torch

import combine_moe_gate_gb300 as M

from gpu_util import status_ok

pytestmark = pytest.mark.gpu

GATE_RTOL, TIE = 6e-6, 2e-6


def scores64(x, score):
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-x))
    top = x.max(1, keepdims=True)
    dead = np.isneginf(top)
    p = np.exp(x - np.where(dead, 0.0, top))
    return np.where(dead, 0.0, p / np.where(dead, 1.0, p.sum(1, keepdims=True)))


def route64(x, bias, k, score, groups, topk_groups, group_top, scale, norm):
    """idx [s, k], gates [s, k] and each token's smallest deciding margin."""
    s, e = x.shape
    sc = scores64(x, score)
    ch = sc + (0.0 if bias is None else bias)
    ch = np.where(np.isneginf(x) | np.isnan(ch), -np.inf, ch)
    idx = np.zeros((s, k), np.int64)
    margin = np.full(s, np.inf)
    for t in range(s):
        allowed = np.ones(e, bool)
        if groups > 1:
            v = np.sort(ch[t].reshape(groups, -1), 1)[:, ::-1][:, :group_top]
            val = np.where(np.isneginf(v[:, 0]), -np.inf, np.where(np.isneginf(v), 0.0, v).sum(1))
            order = sorted(range(groups), key=lambda g: (-val[g], g))
            keep = order[:topk_groups]
            allowed = np.isin(np.arange(e) // (e // groups), keep)
            if topk_groups < groups:
                a, b = val[order[topk_groups - 1]], val[order[topk_groups]]
                if np.isfinite(a) and np.isfinite(b) and a != b:
                    margin[t] = min(margin[t], a - b)
        order = sorted(np.flatnonzero(allowed), key=lambda j: (-ch[t, j], j))
        idx[t] = order[:k]
        c = ch[t, order[:k + 1]]
        gaps = [a - b for a, b in zip(c, c[1:]) if np.isfinite(a) and np.isfinite(b) and a != b]
        margin[t] = min([margin[t]] + gaps)
    g = np.take_along_axis(sc, idx, 1)
    if norm:
        tot = g.sum(1, keepdims=True)
        g = np.where(tot == 0, 0.0, g / np.where(tot == 0, 1.0, tot))
    return idx, g * scale, margin


def run(logits, bias, k, score, groups=1, topk_groups=1, group_top=1, scale=1.0, norm=True):
    s, e = logits.shape
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    idx = torch.full((k, s), -7, dtype=torch.int32, device="cuda")
    gates = torch.full((k, s), -7.0, device="cuda")
    M.moe_route_topk(logits, bias, k, idx, gates, st, score=score, groups=groups, topk_groups=topk_groups,
                     group_top=group_top, scale=scale, flags=M.MOE_FLAG_NORMALIZE_GATES if norm else 0)
    torch.cuda.synchronize()
    status_ok(st)
    return idx.cpu().numpy().T, gates.cpu().numpy().T


def check(logits, bias, k, score, **kw):
    got_idx, got = run(logits, bias, k, score, **kw)
    full = dict(groups=1, topk_groups=1, group_top=1, scale=1.0, norm=True, **{})
    full.update(kw)
    x = logits.float().cpu().numpy().astype(np.float64)
    b = None if bias is None else bias.cpu().numpy().astype(np.float64)
    idx, gates, margin = route64(x, b, k, score, **full)
    same = (got_idx == idx).all(1)
    assert (same | (margin < TIE)).all(), np.flatnonzero(~same)[:5]
    assert same.mean() > 0.99 or len(same) < 100
    err = np.abs(got[same] - gates[same])
    assert (err <= GATE_RTOL * np.abs(gates[same])).all(), err.max()


CASES = [
    # s, e, k, score, bias, groups, topk_groups, group_top, norm, dtype
    (1, 1, 1, "softmax", False, 1, 1, 1, True, "f32"),
    (1, 256, 8, "sigmoid", True, 8, 4, 2, True, "f32"),
    (2, 8, 8, "softmax", False, 1, 1, 1, False, "bf16"),
    (300, 256, 8, "sigmoid", True, 8, 4, 2, True, "f32"),
    (301, 256, 6, "softmax", False, 8, 3, 1, False, "bf16"),
    (257, 60, 4, "softmax", True, 4, 2, 2, True, "f32"),        # rows off the 16-byte grid
    (130, 33, 5, "sigmoid", True, 1, 1, 1, False, "bf16"),
    (77, 160, 6, "sigmoid", False, 8, 3, 1, True, "bf16"),
    (65, 96, 3, "softmax", True, 32, 5, 2, True, "f32"),        # the most groups, of three
    (40, 1000, 32, "sigmoid", True, 10, 7, 2, True, "f32"),
    (33, 1024, 32, "softmax", False, 1, 1, 1, True, "f32"),
    (50, 24, 2, "sigmoid", True, 24, 9, 2, True, "f32"),        # groups of one expert
    (1500, 64, 2, "softmax", False, 1, 1, 1, True, "bf16"),
    (900, 128, 4, "softmax", False, 4, 2, 1, True, "f32"),
    (20, 512, 10, "sigmoid", True, 16, 4, 2, True, "bf16"),
    # more routes than lanes share a token, and all experts chosen
    (37, 32, 32, "sigmoid", True, 1, 1, 1, True, "f32"),
    (41, 16, 10, "softmax", False, 4, 3, 2, False, "bf16"),
    (29, 64, 32, "softmax", True, 8, 4, 2, True, "bf16"),
    (19, 128, 32, "sigmoid", False, 16, 5, 1, True, "f32"),
    (11, 5, 3, "sigmoid", True, 5, 4, 1, True, "f32"),
]


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(map(str, c)))
def test_route_matches_64_bit(c):
    s, e, k, score, use_bias, groups, tg, gt, norm, dt = c
    g = torch.Generator().manual_seed(s * 1000 + e)
    x = torch.randn((s, e), generator=g) * 2
    bias = torch.randn(e, generator=g).mul_(0.1).cuda() if use_bias else None
    x = x.to(torch.float32 if dt == "f32" else torch.bfloat16).cuda()
    check(x, bias, k, score, groups=groups, topk_groups=tg, group_top=gt, scale=2.5 if use_bias else 1.0,
          norm=norm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_ties_go_to_the_lower_index(score, groups):
    x = torch.zeros((9, 64), device="cuda")
    x[1:, 5::7] = 1.0                          # nine experts tied at the top
    x[2] = -0.0
    check(x, None, 6, score, groups=groups, topk_groups=groups // 2 or 1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups,tg,gt", [(64, 1, 1, 1), (64, 8, 3, 2), (30, 5, 2, 2), (256, 8, 4, 1)])
@pytest.mark.parametrize("norm", [True, False])
def test_masked_experts(score, e, groups, tg, gt, norm):
    g = torch.Generator().manual_seed(e)
    x = torch.randn((64, e), generator=g)
    bias = torch.randn(e, generator=g) * 2     # a masked expert's bias must not bring it back
    x[0] = -float("inf")                       # nothing left: gates 0
    x[1, 1:] = -float("inf")                   # one expert left
    x[2, : e // 2] = -float("inf")
    x[3] = torch.finfo(torch.float32).min      # the type's lowest value is a number, not a mask
    x[4, ::2] = -float("inf")                  # every group half masked
    x[5:, 3] = -float("inf")
    for b in (None, bias.cuda()):
        check(x.cuda(), b, 4, score, groups=groups, topk_groups=tg, group_top=gt, norm=norm)
    idx, gates = run(x.cuda(), None, 4, score, groups=groups, topk_groups=tg, group_top=gt, norm=norm)
    assert (gates[0] == 0).all() and (gates[1, 1:] == 0).all()
    assert gates[1, 0] > 0 and idx[1, 0] == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nan_and_infinity_keep_idx_valid(score):
    x = torch.randn((6, 40), generator=torch.Generator().manual_seed(3))
    x[0, 7] = float("nan")
    x[1] = float("nan")
    x[2, 3] = float("inf")
    x[3, [1, 2]] = torch.tensor([float("nan"), -float("inf")])
    idx, gates = run(x.cuda(), None, 5, score)
    for t in range(6):
        assert len(set(idx[t])) == 5 and idx[t].min() >= 0 and idx[t].max() < 40
    if score == "sigmoid":
        assert np.isfinite(gates[[0, 2, 3]]).all() and 7 not in idx[0] and idx[2, 0] == 3
    else:
        assert np.isnan(gates[[0, 1, 2, 3]]).all() and list(idx[1]) == [0, 1, 2, 3, 4]
    assert np.isnan(gates[1]).all() and np.isfinite(gates[4:]).all()


def test_route_is_reproducible_and_honours_its_stream():
    x = torch.randn((3000, 256), generator=torch.Generator().manual_seed(5)).cuda()
    a = run(x, None, 8, "softmax", groups=8, topk_groups=3, group_top=2)
    side = torch.cuda.Stream()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    idx = torch.empty((8, 3000), dtype=torch.int32, device="cuda")
    gates = torch.empty((8, 3000), device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    M.moe_route_topk(x, None, 8, idx, gates, st, groups=8, topk_groups=3, group_top=2,
                     flags=M.MOE_FLAG_NORMALIZE_GATES, stream=side)
    side.synchronize()
    assert (idx.cpu().numpy().T == a[0]).all() and (gates.cpu().numpy().T == a[1]).all()


def test_route_skips_after_an_error():
    x = torch.zeros((4, 8), device="cuda")
    st = torch.full((1,), M.MOE_ERR_CAPACITY, dtype=torch.int32, device="cuda")
    idx = torch.full((2, 4), -3, dtype=torch.int32, device="cuda")
    gates = torch.full((2, 4), -3.0, device="cuda")
    M.moe_route_topk(x, None, 2, idx, gates, st)
    d = torch.full((4, 8), -3.0, device="cuda")
    M.moe_route_bwd(x, torch.zeros_like(idx), gates, d, st)
    torch.cuda.synchronize()
    assert (idx == -3).all() and (gates == -3).all() and (d == -3).all()


# ---------------------------------------------------------------- backward
def grad64(x, idx, dg, score, scale, norm):
    x = x.double().cpu().requires_grad_()
    dead = torch.isneginf(x).all(1, keepdim=True)
    p = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(torch.where(dead, torch.zeros_like(x), x), 1)
    g = p.gather(1, idx.cpu().t().long())
    if norm:
        g = g / g.sum(1, keepdim=True)
    (g * scale * dg.double().cpu().t()).sum().backward()
    return torch.nan_to_num(torch.where(dead, torch.zeros_like(x), x.grad)).numpy()


def run_bwd(x, idx, dg, score, scale, norm, ddt=torch.float32):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = torch.full(x.shape, float("nan"), dtype=ddt, device="cuda")
    M.moe_route_bwd(x, idx, dg, d, st, score=score, scale=scale,
                    flags=M.MOE_FLAG_NORMALIZE_GATES if norm else 0)
    torch.cuda.synchronize()
    status_ok(st)
    return d.float().cpu().numpy()


@pytest.mark.parametrize("s,e,k", [(1, 1, 1), (1, 256, 8), (5, 7, 7), (300, 60, 4), (129, 256, 8),
                                   (70, 33, 32), (40, 1000, 10), (1000, 64, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dt,ddt", [("f32", "f32"), ("bf16", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
def test_route_bwd_matches_64_bit(s, e, k, score, norm, dt, ddt):
    ty = {"f32": torch.float32, "bf16": torch.bfloat16}
    g = torch.Generator().manual_seed(s + e)
    x = (torch.randn((s, e), generator=g) * 2).to(ty[dt]).cuda()
    idx = torch.rand((s, e), generator=g).argsort(1)[:, :k].t().contiguous().int().cuda()
    dg = torch.randn((k, s), generator=g).cuda()
    got = run_bwd(x, idx, dg, score, 2.5, norm, ty[ddt])
    want = grad64(x, idx, dg, score, 2.5, norm)
    # fp32: every gradient is a difference of terms up to scale |d_gates| with k-term sums
    tol = 2.5 * 2.0 ** -24 * (40 + 4 * k) * dg.abs().max().item() + (2.0 ** -8 * np.abs(want) if ddt == "bf16" else 0)
    assert np.isfinite(got).all() and (np.abs(got - want) <= tol).all(), np.abs(got - want).max()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("norm", [True, False])
def test_route_bwd_matches_differences(score, norm):
    """The gradient of sum(d_gates * gates) against central differences of the
    64-bit forward with the selection held fixed."""
    s, e, k, scale, eps = 6, 12, 3, 1.5, 1e-5
    g = torch.Generator().manual_seed(9)
    x = torch.randn((s, e), generator=g)
    dg = torch.randn((k, s), generator=g)
    idx = torch.rand((s, e), generator=g).argsort(1)[:, :k].t().contiguous().int()
    got = run_bwd(x.cuda(), idx.cuda(), dg.cuda(), score, scale, norm)

    def value(v):
        p = np.take_along_axis(scores64(v, score), idx.numpy().T, 1)
        if norm:
            p = p / p.sum(1, keepdims=True)
        return (p * scale * dg.numpy().T).sum()

    x64 = x.double().numpy()
    for t in range(s):
        for j in range(e):
            hi, lo = x64.copy(), x64.copy()
            hi[t, j] += eps
            lo[t, j] -= eps
            # differences: O(eps^2) truncation and 1e-16 / eps cancellation, both below 1e-9; fp32 above
            assert abs((value(hi) - value(lo)) / (2 * eps) - got[t, j]) <= 2e-5


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("norm", [True, False])
def test_route_bwd_masked_rows(score, norm):
    x = torch.randn((4, 16), generator=torch.Generator().manual_seed(2))
    x[0] = -float("inf")
    x[1, 3:] = -float("inf")
    x[2, 0] = torch.finfo(torch.float32).min
    idx = torch.tensor([[0, 1, 2]] * 4, dtype=torch.int32).t().contiguous().cuda()
    dg = torch.ones((3, 4), device="cuda") * torch.tensor([1.0, 2.0, -1.0], device="cuda")[:, None]
    got = run_bwd(x.cuda(), idx, dg, score, 1.0, norm)
    assert np.isfinite(got).all() and (got[0] == 0).all() and (got[1, 3:] == 0).all()
    want = grad64(x, idx, dg, score, 1.0, norm)
    assert (np.abs(got - want) <= 1e-5).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_bwd_of_one_renormalised_route_is_zero(score):
    """The gate is 1 whatever the logit: no rounding error may stand for a gradient."""
    g = torch.Generator().manual_seed(4)
    x, dg = torch.randn((300, 24), generator=g).cuda(), torch.randn((1, 300), generator=g).cuda()
    idx = torch.randint(0, 24, (1, 300), generator=g, dtype=torch.int32).cuda()
    assert (run_bwd(x, idx, dg, score, 2.5, True) == 0).all()
    assert (run_bwd(x[:, :1].contiguous(), torch.zeros_like(idx), dg, "softmax", 2.5, False) == 0).all()


def test_route_bwd_reports_a_bad_index():
    x = torch.zeros((4, 8), device="cuda")
    idx = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
    for bad in (8, -1):
        idx[1, 2] = bad
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        M.moe_route_bwd(x, idx, torch.ones((2, 4), device="cuda"), torch.empty((4, 8), device="cuda"), st)
        torch.cuda.synchronize()
        assert int(st.item()) == M.MOE_ERR_INVALID_ARG
