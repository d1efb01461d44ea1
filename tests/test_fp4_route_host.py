"""moe_route_* and the 4-bit entry points on the host: sizes, argument checks of
the C ABI and of the binding.  Nothing here reaches a launch."""

import ctypes

import pytest
import torch

import combine_moe_gate_gb300 as M

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses are only safe without a GPU")
A, B, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000), ctypes.c_void_p(0x30004)
INV, UNS = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED


def caller(fn, good):
    def call(**kw):
        a = list(good)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return fn(*a)
    return call


@pytest.mark.parametrize("fmt,blk", [("mx", 32), ("nv", 16)])
def test_scale_bytes(fmt, blk):
    lib = M.load()
    for rows, cols in ((1, 32), (128, 128), (129, 160), (300, 2080), (7, 16384), (2048, 4096)):
        want = -(-rows // 128) * -(-(cols // blk) // 4) * 512
        assert M.moe_fp4_scale_bytes(fmt, rows, cols) == want
        assert lib.moe_fp4_scale_bytes(M.FP4[fmt], rows, cols) == want
    for rows, cols in ((0, 32), (1, 0), (1, 48), (-1, 32), (1, -32)):
        assert M.moe_fp4_scale_bytes(fmt, rows, cols) == 0
        assert lib.moe_fp4_scale_bytes(M.FP4[fmt], rows, cols) == 0
    assert lib.moe_fp4_scale_bytes(2, 1, 32) == 0
    with pytest.raises(ValueError, match="fmt"):
        M.moe_fp4_scale_bytes("fp4", 1, 32)


def test_ffn_workspace_size():
    f = M.moe_expert_ffn_fp4_workspace_size
    assert f("mx", "gelu", 2, 10, 64, 96) == 1024 + 1024      # 960 bytes of codes, 2 x 512 of scales
    assert f("nv", "swiglu", 2, 10, 64, 96) == 1024 + 2048
    assert f("nv", "gelu", 1, 1, 48, 96) == 0 and f("nv", "gelu", 1, 1, 64, 40) == 0
    assert f("nv", "gelu", 0, 1, 64, 96) == 0 and f("nv", 7, 1, 1, 64, 96) == 0


@no_gpu
def test_route_refuses():
    lib = M.load()
    before = M.launch_count()
    # logits, ldt, bias, s, e, k, score, groups, topk_groups, group_top, scale, flags, idx, gates, status, stream
    f = caller(lib.moe_route_topk, (A, M.MOE_F32, B, 10, 64, 8, 1, 8, 4, 2, 1.0, 1, A, B, A, None))
    for bad in (dict(a0=None), dict(a0=ODD), dict(a1=2), dict(a2=ODD), dict(a3=0), dict(a4=0), dict(a4=2000),
                dict(a5=0), dict(a5=65), dict(a5=33), dict(a6=2), dict(a7=0), dict(a7=7), dict(a7=128), dict(a8=0),
                dict(a8=9), dict(a9=0), dict(a9=3), dict(a10=float("nan")), dict(a11=2), dict(a11=8), dict(a12=None),
                dict(a13=None), dict(a14=None), dict(a12=ctypes.c_void_p(0x10002))):
        assert f(**bad) == INV, bad
    assert f(a5=9, a8=1) == INV                     # 9 of a group of 8
    assert f(a4=128, a7=64) == UNS                  # more than 32 groups
    g = caller(lib.moe_route_bwd, (A, M.MOE_BF16, A, B, 10, 64, 8, 0, 1.0, 0, A, M.MOE_F32, A, None))
    for bad in (dict(a0=None), dict(a1=3), dict(a2=None), dict(a3=None), dict(a4=0), dict(a5=0), dict(a6=0),
                dict(a7=5), dict(a8=float("nan")), dict(a9=4), dict(a10=None), dict(a10=ODD), dict(a11=2),
                dict(a12=None)):
        assert g(**bad) == INV, bad
    assert M.launch_count() == before


@no_gpu
def test_fp4_conversions_refuse():
    lib = M.load()
    before = M.launch_count()
    # src, sdt, batches, rows, cols, fmt, global, counts, c_dev, q, scale, status, stream
    f = caller(lib.moe_quantize_fp4, (A, M.MOE_BF16, 2, 10, 64, 1, B, A, B, A, B, A, None))
    for bad in (dict(a0=None), dict(a0=ODD), dict(a1=7), dict(a2=0), dict(a3=0), dict(a3=1 << 31), dict(a4=48),
                dict(a4=0), dict(a5=2), dict(a5=0), dict(a6=ctypes.c_void_p(0x10002)), dict(a7=None), dict(a8=None),
                dict(a9=None), dict(a9=ODD), dict(a10=None), dict(a11=None), dict(a2=1 << 31)):
        assert f(**bad) == INV, bad                 # a5=0: MX takes no factor
    # q, scale, batches, rows, cols, fmt, global, counts, c_dev, dst, ddt, status, stream
    g = caller(lib.moe_dequantize_fp4, (A, B, 2, 10, 64, 0, None, None, None, A, M.MOE_F32, A, None))
    for bad in (dict(a0=None), dict(a1=None), dict(a2=0), dict(a3=0), dict(a4=33), dict(a5=3), dict(a6=B), dict(a7=A),
                dict(a9=None), dict(a9=ODD), dict(a10=2), dict(a11=None)):
        assert g(**bad) == INV, bad
    assert M.launch_count() == before


@no_gpu
def test_fp4_products_refuse():
    lib = M.load()
    before = M.launch_count()
    # a_q, a_scale, a_global, counts, c_dev, b_q, b_scale, b_global, bias, fmt, e, c_max, k, n, out, status, stream
    f = caller(lib.moe_product_fp4, (A, B, None, A, B, A, B, None, A, 1, 4, 100, 64, 40, A, B, None))
    for bad in (dict(a0=None), dict(a1=ODD), dict(a2=ctypes.c_void_p(0x10001)), dict(a3=None), dict(a4=None),
                dict(a5=ODD), dict(a6=None), dict(a8=ODD), dict(a9=2), dict(a10=0), dict(a10=1025), dict(a11=0),
                dict(a12=40), dict(a12=0), dict(a13=0), dict(a13=12), dict(a14=None), dict(a14=ODD), dict(a15=None)):
        assert f(**bad) == INV, bad
    assert f(a9=0, a2=A) == INV and f(a9=0, a7=A) == INV        # MX takes no factors
    assert f(a10=1024, a11=1 << 21) == UNS                      # rows beyond 32-bit coordinates
    n = M.moe_expert_ffn_fp4_workspace_size("nv", "gelu", 4, 100, 64, 96)
    good = [A, B, None, None, A, B, A, B, None, A, None, None, None, A, B, None, B, 1, 1, 4, 100, 64, 96, A, n, A, B, None]
    g = caller(lib.moe_expert_ffn_fp4, good)
    for bad in (dict(a0=None), dict(a1=None), dict(a4=None), dict(a5=None), dict(a6=None), dict(a7=ODD), dict(a9=ODD),
                dict(a10=A), dict(a11=A), dict(a12=A), dict(a13=None), dict(a14=None), dict(a16=ODD), dict(a17=3),
                dict(a18=5), dict(a19=0), dict(a20=0), dict(a21=40), dict(a22=40), dict(a23=None), dict(a24=n - 1),
                dict(a25=None), dict(a26=None), dict(a2=ctypes.c_void_p(0x10002))):
        assert g(**bad) == INV, bad
    assert g(a18=2) == INV                                      # SwiGLU without w3
    assert g(a18=2, a10=A, a11=B) == INV                        # SwiGLU with biases
    assert M.launch_count() == before


@no_gpu
def test_binding_refuses(monkeypatch):
    monkeypatch.setattr(M, "_on_device", lambda t: True)
    before = M.launch_count()
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    route = lambda **kw: M.moe_route_topk(**{**dict(logits=torch.zeros(10, 8), bias=None, k=2, idx=i32(2, 10),
                                                    gates=torch.zeros(2, 10), dev_status=i32(1)), **kw})
    with pytest.raises(ValueError, match="score"):
        route(score="tanh")
    with pytest.raises(ValueError, match="idx: shape"):
        route(idx=i32(10, 2))
    with pytest.raises(ValueError, match="bias: shape"):
        route(bias=torch.zeros(9))
    with pytest.raises(TypeError, match="unsupported dtype"):
        route(logits=torch.zeros(10, 8, dtype=torch.float16))
    with pytest.raises(ValueError, match="logits: must be contiguous"):
        route(logits=torch.zeros(10, 16)[:, :8])
    with pytest.raises(ValueError, match="d_logits: shape"):
        M.moe_route_bwd(torch.zeros(10, 8), i32(2, 10), torch.zeros(2, 10), torch.zeros(8, 10), i32(1))
    x = torch.zeros(2, 10, 64, dtype=torch.bfloat16)
    ok = dict(src=x, fmt="nv", q=u8(2, 10, 32), scale=u8(2, M.moe_fp4_scale_bytes("nv", 10, 64)), dev_status=i32(1))
    for kw, what in ((dict(q=u8(2, 10, 64)), "q: shape"), (dict(scale=u8(2, 100)), "scale: shape"),
                     (dict(global_scale=torch.zeros(3)), "global_scale: shape"), (dict(counts=i32(3)), "counts: shape"),
                     (dict(fmt="e2m1"), "fmt")):
        with pytest.raises(ValueError, match=what):
            M.moe_quantize_fp4(**{**ok, **kw})
    with pytest.raises(TypeError, match="q: dtype"):
        M.moe_quantize_fp4(**{**ok, "q": torch.zeros(2, 10, 32, dtype=torch.int8)})
    n = lambda r, c: M.moe_fp4_scale_bytes("mx", r, c)
    prod = dict(a_q=u8(2, 10, 32), a_scale=u8(2, n(10, 64)), a_global=None, counts=i32(2), c_dev=i32(1),
                b_q=u8(2, 24, 32), b_scale=u8(2, n(24, 64)), b_global=None, bias=None, fmt="mx",
                out=torch.zeros(2, 10, 24, dtype=torch.bfloat16), dev_status=i32(1))
    for kw, what in ((dict(b_q=u8(2, 24, 16)), "b_q: shape"), (dict(a_scale=u8(2, 1)), "a_scale: shape"),
                     (dict(bias=torch.zeros(2, 10, dtype=torch.bfloat16)), "bias: shape")):
        with pytest.raises(ValueError, match=what):
            M.moe_product_fp4(**{**prod, **kw})
    assert M.launch_count() == before
