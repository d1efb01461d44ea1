"""The reciprocal and quotient of csrc/exact.cuh against CUDA's correctly rounded
ones over the ranges they are stated for."""

import pytest
import torch

import exact_lib

pytestmark = pytest.mark.gpu


def bad_counter():
    return torch.zeros(1, dtype=torch.int64, device="cuda")


def test_rcp_mid_rounds_every_mantissa_correctly():
    """Every float of 2^-120 <= x <= 2^126."""
    bad = bad_counter()
    torch.cuda.synchronize()
    for ex in range(127 - 120, 127 + 126):
        assert exact_lib.load().exact_rcp(ex, 1 << 23, bad.data_ptr()) == 0
    assert exact_lib.load().exact_rcp(127 + 126, 1, bad.data_ptr()) == 0
    torch.cuda.synchronize()
    assert int(bad.item()) == 0


@pytest.mark.parametrize("a,b", [
    ((-100, 0), (0, 10)),       # softmax: an exponential over a sum of up to 1024
    ((-60, 59), (-40, 39)),     # a block's largest magnitude over 6 g
    ((-100, -99), (-10, 20)),   # the smallest numerators
    ((60, 110), (-9, -9)),      # quotients up to 2^120
    ((-60, -50), (50, 59)),     # and down to 2^-120
    ((0, 0), (0, 0)),
], ids=str)
def test_div_mid_rounds_correctly(a, b):
    bad = bad_counter()
    torch.cuda.synchronize()
    for seed in range(4):
        assert exact_lib.load().exact_div(seed, 4096, 64, *a, *b, bad.data_ptr()) == 0   # 67 M pairs each
    torch.cuda.synchronize()
    assert int(bad.item()) == 0
