"""8-bit integer experts where the calls can go wrong: offsets that do not start at 0, hidden rows in GELU's
tail, and scales whose product leaves fp32's range."""

import pytest
import torch

import combine_moe_gate_gb300 as M
import test_gpu_int8 as S

pytestmark = pytest.mark.gpu

BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8
HALF, U = S.HALF, S.U


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


# few rows (dot products: up to 64 of 128 experts) and many (tiles)
@pytest.mark.parametrize("e,rows", [(128, 64), (1, 80)])
def test_gelu_of_a_row_in_the_tail(e, rows):
    """Pre-activations from -8 to -3, exact by construction: the row's maximum lies in the tail as well, so
    the 8-bit step of the hidden does.  The approximation is within 1.3e-4 of the value there, the bf16
    hidden within half a step of that, its code within half a code."""
    m, h, j = 16, 64, e // 3
    x = torch.zeros((rows, m), dtype=I8, device="cuda")
    x[:, 5] = torch.arange(128 - rows, 128, device="cuda")
    sx = torch.full((rows,), 1 / 16, device="cuda")
    w1, w2 = torch.zeros((e, h, m), dtype=I8, device="cuda"), torch.zeros((e, m, h), dtype=I8, device="cuda")
    w1[:, :, 5] = -1
    w2[:, torch.arange(m), torch.arange(m)] = 127
    s1 = (1 - torch.arange(h, device="cuda") / 1024).repeat(e, 1).contiguous()
    s2 = torch.full((e, m), 1 / 127, device="cuda")
    off = None
    if e > 1:
        off = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
        off[j + 1:] = rows
    ws = torch.zeros(M.moe_expert_ffn_int8_workspace_size("gelu", e, rows, m, h), dtype=torch.uint8, device="cuda")
    out, st = torch.zeros((rows, m), dtype=BF, device="cuda"), S.status()
    M.moe_expert_ffn_int8(x, sx, off, w1, s1, None, None, None, w2, s2, None, "gelu", ws, out, st)
    assert st.item() == 0
    a = -x[:, 5, None].double() / 16 * s1[j].double()
    assert a.min() < -7.9 and a.max() < -2.8
    want = 0.5 * a * torch.special.erfc(-a * 0.5 ** 0.5)
    hid = ws[: rows * h * 2].view(BF).view(rows, h)
    rel = HALF[BF] * 1.01 + 1.5e-4
    S.near(hid, want, rel * want.abs(), "hid")
    top = want.abs().amax(1, keepdim=True)
    S.near(out, want[:, :m], 0.5 / 127 * 1.01 * top + (rel + HALF[BF] * 1.01) * want[:, :m].abs(), "out")


# (row scale, channel scale) whose product is subnormal, below the smallest number, too large; and one of each
# beside ordinary ones.  few rows (dot products) and many (tiles)
@pytest.mark.parametrize("sx,sw", [(2.0 ** -70, 1.4 * 2.0 ** -72), (2.0 ** -80, 1.3 * 2.0 ** -76), (2.0 ** 70, 1.7 * 2.0 ** 60),
                                   (2.0 ** 100, 2.0 ** -100), (2.0 ** -107, 2.0 ** -30)])
@pytest.mark.parametrize("n", [2, 90])
@pytest.mark.parametrize("mixed", [False, True])
def test_product_of_scales_far_from_1(sx, sw, n, mixed):
    k, n_out = 512, 136
    a, w = S.codes((n, k), 1), S.codes((1, n_out, k), 2)
    a[n // 2] = 0                                         # 0 times whatever the scales are
    ra = (torch.rand(n, generator=S.gen(3), device="cuda") + 0.5) * sx
    cw = (torch.rand((1, n_out), generator=S.gen(4), device="cuda") + 0.5) * sw
    if mixed:
        ra[1::2] /= sx
        cw[:, ::3] /= sw
    out = S.product(a, ra, None, w, cw, None, F32)
    acc = a.double() @ w[0].double().t()                  # exact: k <= 1024
    want = acc * (ra.double()[:, None] * cw[0].double())
    over = want.abs() >= 2.0 ** 128 * (1 - 2.0 ** -25)    # rounds to an infinity
    assert torch.equal(out.double().isinf(), over)
    bound = 4 * U * want.abs() + 2.0 ** -149              # three roundings, or one to a subnormal number
    S.near(torch.where(over, 0.0, out), torch.where(over, 0.0, want), bound)
    assert (out[n // 2] == 0).all()


@pytest.mark.parametrize("n", [2, 90])
def test_gated_hidden_of_scales_far_from_1(n):
    """silu of a tiny a times a huge b is an ordinary number: a's scales multiply to a subnormal one."""
    m = h = 64
    x, w = S.codes((n, m), 1), S.codes((1, h, m), 2)
    w3, w2 = S.codes((1, h, m), 3), S.codes((1, m, h), 4)
    sx = torch.full((n,), 2.0 ** -70, device="cuda")
    s1 = (torch.rand((1, h), generator=S.gen(5), device="cuda") + 0.5) * 2.0 ** -72
    s3 = (torch.rand((1, h), generator=S.gen(6), device="cuda") + 0.5) * 2.0 ** 110
    s2 = torch.ones((1, m), device="cuda")
    ws = torch.zeros(M.moe_expert_ffn_int8_workspace_size("swiglu", 1, n, m, h), dtype=torch.uint8, device="cuda")
    out, st = torch.zeros((n, m), dtype=BF, device="cuda"), S.status()
    M.moe_expert_ffn_int8(x, sx, None, w, s1, None, w3, s3, w2, s2, None, "swiglu", ws, out, st)
    assert st.item() == 0
    a = x.double() @ w[0].double().t() * (sx.double()[:, None] * s1[0].double())
    b = x.double() @ w3[0].double().t() * (sx.double()[:, None] * s3[0].double())
    want = a / (1 + torch.exp(-a)) * b
    hid = ws[: n * h * 2].view(BF).view(n, h)
    # a: one rounding of 2^-24, or to a subnormal's 2^-150; b: two; silu 8 and its product one
    S.near(hid, want, (HALF[BF] * 1.01 + 16 * U) * want.abs() + 2.0 ** -149 * b.abs(), "hid")


@pytest.mark.parametrize("n", [2, 90])
def test_scales_far_from_1_change_no_other_row_or_channel(n):
    """The same bits beside rows and channels of extreme scales as beside ordinary ones."""
    k, n_out = 528, 136
    a, w = S.codes((n, k), 1), S.codes((1, n_out, k), 2)
    ra = torch.rand(n, generator=S.gen(3), device="cuda") + 0.5
    cw = torch.rand((1, n_out), generator=S.gen(4), device="cuda") + 0.5
    bias = torch.randn((1, n_out), generator=S.gen(5), device="cuda").bfloat16()
    out = S.product(a, ra, None, w, cw, bias, F32)
    ra[::2] *= 2.0 ** -70
    cw[:, 1::3] *= 2.0 ** -75
    far = S.product(a, ra, None, w, cw, bias, F32)
    assert torch.equal(out[1::2, ::3], far[1::2, ::3]) and torch.equal(out[1::2, 2::3], far[1::2, 2::3])
