"""The sorted-row and 8-bit integer entry points on the host: sizes, argument checks of the C ABI and of
the binding.  Nothing here reaches a launch."""

import ctypes
import types

import pytest
import torch

import combine_moe_gate_gb300 as M

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses are only safe without a GPU")
A, B, ODD, ODD4 = (ctypes.c_void_p(x) for x in (0x10000, 0x20000, 0x30004, 0x30002))
INV, UNS, BF, F32 = M.MOE_ERR_INVALID_ARG, M.MOE_ERR_UNSUPPORTED, M.MOE_BF16, M.MOE_F32
RELU, GELU, SWIGLU = 0, 1, 2
BIG = 1 << 60


def check(fn, good, bad, pointers, words=()):
    """fn refuses each (position, value) of bad, NULL and misaligned `pointers` (16 bytes) and `words` (4)."""
    before = M.launch_count()

    def call(i, v):
        a = list(good)
        a[i] = v
        return fn(*a)

    for i, v, want in bad:
        assert call(i, v) == want, (i, v)
    for i in pointers:
        assert call(i, None) == INV and call(i, ODD) == INV, i
    for i in words:
        assert call(i, None) == INV and call(i, ODD4) == INV, i
    assert M.launch_count() == before


def test_workspace_sizes():
    assert M.moe_sort_workspace_size(65536, 64, 2) >= 65 * 128 * 4
    assert M.moe_sort_workspace_size(1, 1, 1) >= 8
    for s, e, k in ((0, 4, 1), (5, 0, 1), (5, 1025, 1), (5, 4, 0), (5, 40, 33), (1 << 40, 4, 2)):
        assert M.moe_sort_workspace_size(s, e, k) == 0
    # d_pre, and 64-row blocks of four operands an expert
    assert M.moe_expert_ffn_sorted_bwd_workspace_size("gelu", 4, 1000, 64, 96) >= 1000 * 96 * 2 + 4 * 64 * (2 * 64 + 2 * 96) * 2
    assert M.moe_expert_ffn_sorted_bwd_workspace_size("gelu", 4, 1000, 60, 96) == 0
    assert M.moe_expert_ffn_sorted_bwd_workspace_size(7, 4, 1000, 64, 96) == 0
    assert M.moe_product_int8_workspace_size(4, 1000, 64, 96) >= 1000 * 64 * 2
    assert M.moe_product_int8_workspace_size(4, 8, 64, 96) > 0
    for e, n, k, no in ((0, 9, 64, 8), (4, 0, 64, 8), (4, 9, 24, 8), (4, 9, 64, 12), (4, 9, 1 << 17, 8)):
        assert M.moe_product_int8_workspace_size(e, n, k, no) == 0
    assert M.moe_expert_ffn_int8_workspace_size("relu", 4, 100, 64, 96) >= 100 * (96 * 4 + 4 + 64 * 2)
    assert M.moe_expert_ffn_int8_workspace_size("relu", 4, 100, 72, 96) == 0


@no_gpu
def test_products_leave_room_for_the_last_channel_tile():
    """Channels are counted in 32 bits, and the last tile of them reaches past the end."""
    for e, no in ((1, 2 ** 31 - 8), (1, 2 ** 31 - 256), (4, 2 ** 29 - 8)):
        assert M.moe_product_int8_workspace_size(e, 8, 16, no) == 0
    assert M.moe_product_int8_workspace_size(1, 8, 16, 2 ** 31 - 1024) > 0


def test_sort_refuses():
    good = (A, 100, 8, 2, A, A, None, A, BIG, A, None)     # idx s e k rows offsets source ws bytes status stream
    check(M.load().moe_sort_routes, good,
          [(1, 0, INV), (1, 1 << 31, INV), (2, 0, INV), (2, 1025, INV), (3, 0, INV), (3, 33, INV), (6, ODD4, INV),
           (8, 8, INV)], pointers=(7,), words=(0, 4, 5, 9))


@no_gpu
def test_movements_refuse():
    lib = M.load()
    dims = lambda o: [(o, 0, INV), (o + 1, 0, INV), (o + 1, 60, INV), (o + 2, 0, INV), (o + 2, 33, INV), (o + 3, 0, INV),
                      (o + 3, 1 << 31, INV), (1, 7, INV)]
    # x dt rows gates | s m k n | out status stream
    good = (A, BF, A, A, 100, 64, 2, 200, B, A, None)
    for fn in (lib.moe_encode_sorted, lib.moe_decode_sorted):
        check(fn, good, dims(4) + [(3, ODD4, INV)], pointers=(0, 8), words=(2, 9))
    # read read dt rows gates | s m k n | out d_gates status stream
    good = (A, B, BF, A, A, 100, 64, 2, 200, B, A, A, None)
    d = [(i, v, w) if i != 1 else (2, v, w) for i, v, w in dims(5)]
    check(lib.moe_decode_sorted_bwd, good, d, pointers=(0, 1, 9), words=(3, 4, 10, 11))
    # d_gates need the gates and x
    check(lib.moe_encode_sorted_bwd, good, d + [(4, None, INV), (1, None, INV), (10, ODD4, INV)], pointers=(0, 9),
          words=(3, 11))


@no_gpu
def test_sorted_mlp_refuses():
    lib = M.load()
    # x dt off w1 b1 w3 w2 b2 act e n m h hid pre out status stream
    good = (A, BF, A, A, A, None, A, A, GELU, 4, 100, 64, 96, B, None, B, A, None)
    check(lib.moe_expert_ffn_sorted, good,
          [(1, 7, INV), (1, F32, UNS), (4, ODD, INV), (7, ODD, INV), (8, 3, INV), (9, 0, INV), (9, 1025, INV), (10, 0, INV),
           (10, 1 << 31, UNS), (11, 0, INV), (11, 60, INV), (12, 100, INV), (14, ODD, INV), (12, 1 << 30, UNS)],
          pointers=(0, 3, 6, 13, 15), words=(2, 16))
    sw = list(good)
    sw[8] = SWIGLU
    assert lib.moe_expert_ffn_sorted(*sw) == INV            # no w3, and biases
    # x hid pre dt off w1 w3 w2 act e n m h d_out ws bytes d_x wdt dw1 dw3 dw2 db1 db2 status stream
    good = (A, A, A, BF, A, A, None, A, GELU, 4, 100, 64, 96, A, A, BIG, B, BF, B, None, B, B, B, A, None)
    check(lib.moe_expert_ffn_sorted_bwd, good,
          [(3, F32, UNS), (3, 5, INV), (17, 5, INV), (8, -1, INV), (9, 0, INV), (10, 0, INV), (11, 4, INV), (12, 4, INV),
           (15, 1000, INV), (21, ODD, INV), (22, ODD, INV)], pointers=(0, 1, 2, 5, 7, 13, 14, 16, 18, 20), words=(4, 23))
    sw = list(good)
    sw[8] = SWIGLU
    assert lib.moe_expert_ffn_sorted_bwd(*sw) == INV


@no_gpu
def test_int8_refuses():
    lib = M.load()
    # src dt rows s cols k n q scale status stream
    good = (A, BF, None, 100, 64, 0, 100, B, B, A, None)
    check(lib.moe_quantize_rows_int8, good,
          [(1, 7, INV), (3, 0, INV), (4, 0, INV), (4, 24, INV), (5, 1, INV), (6, 99, INV), (6, 0, INV)], pointers=(0, 7),
          words=(8, 9))
    fan = (A, BF, A, 100, 64, 2, 250, B, B, A, None)
    check(lib.moe_quantize_rows_int8, fan, [(2, ODD4, INV), (5, 0, INV), (5, 33, INV), (6, 0, INV)], pointers=(0, 7))
    # a sa off b sb bias e n k n_out ws bytes out odt status stream
    good = (A, A, A, A, A, None, 4, 100, 64, 96, A, BIG, B, BF, A, None)
    check(lib.moe_product_int8, good,
          [(2, None, INV), (2, ODD4, INV), (5, ODD, INV), (6, 0, INV), (6, 1025, INV), (7, 0, INV), (8, 0, INV), (8, 24, INV),
           (8, 1 << 17, UNS), (9, 0, INV), (9, 12, INV), (9, 1 << 30, UNS), (11, 1000, INV), (13, 9, INV), (7, 1 << 31, UNS)],
          pointers=(0, 3, 10, 12), words=(1, 4, 14))
    # x sx off w1 s1 b1 w3 s3 w2 s2 b2 act e n m h ws bytes out status stream
    good = (A, A, A, A, A, None, None, None, A, A, None, GELU, 4, 100, 64, 96, A, BIG, B, A, None)
    check(lib.moe_expert_ffn_int8, good,
          [(2, None, INV), (5, ODD, INV), (6, A, INV), (7, A, INV), (11, 3, INV), (11, SWIGLU, INV), (12, 0, INV), (13, 0, INV),
           (14, 24, INV), (15, 24, INV), (14, 1 << 17, UNS), (17, 1000, INV)], pointers=(0, 3, 8, 16, 18),
          words=(1, 4, 9, 19))


@no_gpu
def test_binding_refuses(monkeypatch):
    monkeypatch.setattr(M, "_on_device", lambda t: True)
    i32, f32, bf, i8 = torch.int32, torch.float32, torch.bfloat16, torch.int8
    z = lambda *shape, dt=f32: torch.zeros(shape, dtype=dt)
    st, ws = z(1, dt=i32), z(1 << 20, dt=torch.uint8)
    before = M.launch_count()
    with pytest.raises(ValueError, match="offsets: shape"):
        M.moe_sort_routes(z(2, 9, dt=i32), 4, z(2, 9, dt=i32), z(4, dt=i32), ws, st)
    with pytest.raises(TypeError, match="idx: dtype"):
        M.moe_sort_routes(z(2, 9, dt=torch.int64), 4, z(2, 9, dt=i32), z(5, dt=i32), ws, st)
    with pytest.raises(ValueError, match="source: shape"):
        M.moe_sort_routes(z(2, 9, dt=i32), 4, z(2, 9, dt=i32), z(5, dt=i32), ws, st, source=z(17, dt=i32))
    rows = z(2, 9, dt=i32)
    with pytest.raises(ValueError, match="x: shape"):
        M.moe_encode_sorted(z(8, 64, dt=bf), rows, z(18, 64, dt=bf), st)
    with pytest.raises(TypeError, match="out: dtype"):
        M.moe_encode_sorted(z(9, 64, dt=bf), rows, z(18, 64), st)
    with pytest.raises(TypeError, match="unsupported dtype"):
        M.moe_encode_sorted(z(9, 64, dt=torch.float16), rows, z(18, 64, dt=torch.float16), st)
    with pytest.raises(ValueError, match="must be contiguous"):
        M.moe_decode_sorted(z(18, 128, dt=bf)[:, :64], rows, z(9, 64, dt=bf), st)
    with pytest.raises(ValueError, match="gates: shape"):
        M.moe_decode_sorted(z(18, 64, dt=bf), rows, z(9, 64, dt=bf), st, gates=z(9, 2))
    with pytest.raises(ValueError, match="d_gates: shape"):
        M.moe_decode_sorted_bwd(z(9, 64, dt=bf), z(18, 64, dt=bf), rows, z(2, 9), z(18, 64, dt=bf), z(2, 8), st)
    nul = types.SimpleNamespace(cuda_stream=0)
    with pytest.raises(M.MoEError):
        M.moe_encode_sorted_bwd(z(18, 64, dt=bf), rows, z(9, 64, dt=bf), st, d_gates=z(2, 9), stream=nul)
    w1, w2 = z(4, 96, 64, dt=bf), z(4, 64, 96, dt=bf)
    with pytest.raises(ValueError, match="pre: shape"):
        M.moe_expert_ffn_sorted(z(18, 64, dt=bf), z(5, dt=i32), w1, None, w1, w2, None, "swiglu", z(18, 96, dt=bf),
                                z(18, 64, dt=bf), st, pre=z(18, 96, dt=bf))
    with pytest.raises(ValueError, match="q: shape"):
        M.moe_quantize_rows_int8(z(9, 64), z(9, 32, dt=i8), z(9), st)
    with pytest.raises(ValueError, match="scale: shape"):
        M.moe_quantize_rows_int8(z(9, 64), z(18, 64, dt=i8), z(9), st, rows=rows)
    with pytest.raises(TypeError, match="b_q: dtype"):
        M.moe_product_int8(z(18, 64, dt=i8), z(18), z(5, dt=i32), z(4, 96, 64), z(4, 96), None, ws, z(18, 96), st)
    with pytest.raises(ValueError, match="b_scale: shape"):
        M.moe_product_int8(z(18, 64, dt=i8), z(18), z(5, dt=i32), z(4, 96, 64, dt=i8), z(4, 64), None, ws, z(18, 96), st)
    with pytest.raises(M.MoEError):
        M.moe_product_int8(z(18, 64, dt=i8), z(18), None, z(4, 96, 64, dt=i8), z(4, 96), None, ws, z(18, 96), st,
                           stream=nul)
    assert M.launch_count() == before
