"""moe_route_topk against its definition in fp32, bit for bit: the scores' single
operations (CUDA's expf, correctly rounded divisions, the softmax sum by adjacent
pairs over the padded width), the choices, the groups and the order, on logits
full of ties and near ties and on rows that cross the switches between the
quotient's forms (exponentials below 2^-100, a sigmoid's 1 + exp(-l) above 2^126)."""

import pytest
import torch

import combine_moe_gate_gb300 as M

import exact_lib
from gpu_util import bits, status_ok

pytestmark = pytest.mark.gpu

NEG = -float("inf")


def scores32(x, score):
    if score == "sigmoid":
        t = 1.0 + exact_lib.expf(-x)
        return torch.ones_like(t) / t
    top = x.amax(1, keepdim=True)
    p = exact_lib.expf(x - torch.where(top == NEG, torch.zeros_like(top), top))
    t = torch.nn.functional.pad(p, (0, (1 << (x.shape[1] - 1).bit_length()) - x.shape[1]))
    while t.shape[1] > 1:
        t = t[:, 0::2] + t[:, 1::2]
    return torch.where(t == 0, torch.zeros_like(p), p / t)


def descending(v):
    return torch.sort(v, dim=1, descending=True, stable=True)[1]


def route32(logits, bias, k, score, groups, topk_groups, group_top, scale, norm):
    x = logits.float()
    s, e = x.shape
    sc = scores32(x, score)
    ch = sc if bias is None else sc + bias
    ch = torch.where((x == NEG) | ch.isnan(), torch.full_like(ch, NEG), ch)
    order = descending(ch)
    if groups > 1:
        best = ch.view(s, groups, -1).sort(2, descending=True)[0]
        val = best[..., 0]
        if group_top == 2 and e > groups:
            val = torch.where(best[..., 1] > NEG, val + best[..., 1], val)
        keep = torch.zeros((s, groups), dtype=torch.int32, device=x.device)
        keep.scatter_(1, descending(val)[:, :topk_groups], 1)
        inside = keep.repeat_interleave(e // groups, 1).gather(1, order)
        order = order.gather(1, descending(inside))
    idx = order[:, :k]
    g = sc.gather(1, idx)
    if norm:
        total = torch.zeros_like(g[:, 0])
        for r in range(k):
            total = total + g[:, r]
        g = torch.where(total[:, None] == 0, torch.zeros_like(g), g / total[:, None])
    return idx.t().int().contiguous(), (g * scale).t().contiguous()


def logits_of(kind, s, e, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "random":
        x = torch.randn((s, e), generator=g) * 2
    elif kind == "ties":          # a few values only
        x = torch.randint(-3, 4, (s, e), generator=g) * 0.5
    elif kind == "near":          # neighbours a few units in the last place apart
        x = torch.randn((s, 1), generator=g).expand(s, e).contiguous()
        x = (x.view(torch.int32) + torch.randint(-6, 7, (s, e), generator=g, dtype=torch.int32)).view(torch.float32)
    else:                         # "wide": across every switch and underflow, some experts masked
        x = torch.rand((s, e), generator=g) * -115.0 + torch.randint(0, 8, (s, 1), generator=g)
        x[torch.rand((s, e), generator=g) < 0.1] = NEG
    return x.to(dtype).cuda()


SHAPES = [
    # s, e, k, groups, topk_groups, group_top
    (400, 5, 3, 1, 1, 1),
    (300, 16, 16, 4, 4, 2),
    (300, 33, 7, 1, 1, 1),
    (500, 60, 4, 4, 2, 2),
    (500, 64, 2, 1, 1, 1),
    (300, 64, 32, 8, 4, 1),
    (200, 96, 6, 32, 9, 2),
    (200, 128, 8, 4, 2, 2),
    (200, 160, 6, 8, 3, 1),
    (300, 256, 8, 8, 4, 2),
    (200, 256, 32, 1, 1, 1),
    (100, 384, 9, 3, 2, 2),
    (100, 512, 10, 16, 4, 2),
    (60, 1000, 32, 10, 7, 1),
    (60, 1024, 8, 1, 1, 1),
]


@pytest.mark.parametrize("kind", ["random", "ties", "near", "wide"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda c: "-".join(map(str, c)))
def test_route_is_its_fp32_definition_bit_for_bit(kind, score, shape):
    s, e, k, groups, tg, gt = shape
    for dtype in (torch.float32, torch.bfloat16):
        x = logits_of(kind, s, e, dtype, s + e)
        for norm, with_bias in ((True, False), (False, True), (True, True)):
            bias = None
            if with_bias:   # few distinct values: sums tie as well
                bias = (torch.randint(-2, 3, (e,), generator=torch.Generator().manual_seed(e)) * 0.03125).cuda()
            idx = torch.full((k, s), -7, dtype=torch.int32, device="cuda")
            gates = torch.full((k, s), -7.0, device="cuda")
            st = torch.zeros(1, dtype=torch.int32, device="cuda")
            M.moe_route_topk(x, bias, k, idx, gates, st, score=score, groups=groups, topk_groups=tg, group_top=gt,
                             scale=2.5, flags=M.MOE_FLAG_NORMALIZE_GATES if norm else 0)
            torch.cuda.synchronize()
            status_ok(st)
            want_idx, want = route32(x, bias, k, score, groups, tg, gt, 2.5, norm)
            assert torch.equal(idx, want_idx), (dtype, norm, with_bias)
            assert (bits(gates) == bits(want)).all(), (dtype, norm, with_bias)
