"""GB300-native top-k MoE layer hot path: Python binding of libmoe_gate.so.

Every step runs in the CUDA library (include/moe_gate.h); this module only
marshals torch tensors into the C ABI: data pointers, sizes taken from the
tensor shapes, the current CUDA stream.  There is no fallback: if the library
is missing, importing the entry points raises.

Functions keep the C names:
    moe_gate_topk, moe_capacity_locations, moe_capacity_locations_noalloc,
    moe_encode, moe_expert_ffn,
    moe_decode, moe_decode_bwd, moe_encode_bwd, moe_layer_forward, moe_gate_bwd,
    moe_route_topk, moe_route_bwd,
    moe_quantize_fp4, moe_dequantize_fp4, moe_product_fp4, moe_expert_ffn_fp4
plus the size queries and `MoEError`.
"""

import ctypes
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libmoe_gate.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "moe_gate.h")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_CUDA, MOE_ERR_CAPACITY, MOE_ERR_TIMEOUT = range(6)
MOE_F32, MOE_BF16 = 0, 1
ACT = {"relu": 0, "gelu": 1, "swiglu": 2}
SCORE = {"softmax": 0, "sigmoid": 1}
FP4 = {"mx": 0, "nv": 1}
MOE_FLAG_NORMALIZE_GATES = 1
MOE_FLAG_ZERO_FILL = 2

_lib = None


class MoEError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__(f"{where}: {status_str(code)} ({code})")


def load():
    """Load libmoe_gate.so (build it first with combine_moe_gate_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing "
                           "(run `python -m combine_moe_gate_gb300.build`)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, I64, U, F, SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint,
                           ctypes.c_float, ctypes.c_size_t)
    sigs = {
        "moe_gate_topk": (I, [P, I, P, P, I64, I, I, I, U, P, P, P, P]),
        "moe_gate_bwd": (I, [P, I, P, P, I64, I, I, I, U, P, P, P, P, P, P, P, P, P]),
        "moe_capacity_bound": (I64, [F, I64, I, I]),
        "moe_capacity_workspace_size": (SZ, [I64, I, I]),
        "moe_capacity_locations": (I, [P, I64, I, I, F, I64, P, SZ, P, P, P, P, P]),
        "moe_capacity_locations_noalloc": (I, [P, I64, I, I, F, I64, P, P, P, P, P]),
        "moe_encode": (I, [P, I, P, P, P, P, I64, I, I, I, I64, U, P, P, P]),
        "moe_expert_ffn_workspace_size": (SZ, [I, I, I, I64, I, I]),
        "moe_expert_ffn": (I, [P, I, P, P, P, P, P, P, P, I, I, I64, I, I, P, SZ, P, P, P]),
        "moe_expert_ffn_train": (I, [P, I, P, P, P, P, P, P, P, I, I, I64, I, I, P, SZ, P, P, P, P]),
        "moe_expert_ffn_bwd_workspace_size": (SZ, [I, I, I, I64, I, I]),
        "moe_expert_ffn_bwd": (I, [P, P, I, P, P, P, P, P, P, I, I, I64, I, I, P, P, SZ, P, P, P,
                                   P, P, P, P, P]),
        "moe_expert_ffn_bwd_saved": (I, [P, P, P, I, P, P, P, P, P, I, I, I64, I, I, P, P, SZ, P, I,
                                         P, P, P, P, P, P, P]),
        "moe_decode": (I, [P, I, P, P, P, P, I64, I, I, I, I64, P, P, P]),
        "moe_decode_bwd": (I, [P, P, I, P, P, P, P, P, I64, I, I, I, I64, U, P, P, P, P]),
        "moe_encode_bwd": (I, [P, I, P, P, P, I64, I, I, I, I64, P, P, P]),
        "moe_layer_workspace_size": (SZ, [I, I, I64, I, I, I, I64, I]),
        "moe_layer_forward": (I, [P, I, P, P, P, P, P, P, P, I, I64, I, I, I, I, F, I64, U,
                                  P, P, P, P, P, P, P, P, P, SZ, P, P]),
        "moe_layer_forward_host": (I, [P, P, P, I, P, P, P, P, P, P, P, I, I64, I, I, I, I, F, I64,
                                       U, P, P, P, P, P, P, P, P, P, SZ, P, P]),
        "moe_layer_forward_pipelined": (I, [P, I, P, P, P, P, P, P, P, I, I64, I, I, I, I, F, I64,
                                            U, P, P, P, P, P, P, P, P, P, SZ, P, I, P, P, P]),
        "moe_probe_fp32_fma": (I, [I, I, I, P, P]),
        "moe_quantize_rows_fp8": (I, [P, I64, I64, I, P, P, P, P, P, P]),
        "moe_expert_ffn_fp8_workspace_size": (SZ, [I, I64, I, I]),
        "moe_expert_ffn_fp8": (I, [P, P, P, P, P, P, P, P, P, P, I, I, I64, I, I, P, SZ, P, P, P]),
        "moe_route_topk": (I, [P, I, P, I64, I, I, I, I, I, I, F, U, P, P, P, P]),
        "moe_route_bwd": (I, [P, I, P, P, I64, I, I, I, F, U, P, I, P, P]),
        "moe_fp4_scale_bytes": (SZ, [I, I64, I]),
        "moe_quantize_fp4": (I, [P, I, I64, I64, I, I, P, P, P, P, P, P, P]),
        "moe_dequantize_fp4": (I, [P, P, I64, I64, I, I, P, P, P, P, I, P, P]),
        "moe_product_fp4": (I, [P, P, P, P, P, P, P, P, P, I, I, I64, I, I, P, P, P]),
        "moe_expert_ffn_fp4_workspace_size": (SZ, [I, I, I, I64, I, I]),
        "moe_expert_ffn_fp4": (I, [P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, I, I, I, I64, I,
                                   I, P, SZ, P, P, P]),
        "moe_status_str": (ctypes.c_char_p, [I]),
        "moe_launch_count": (ctypes.c_uint64, []),
        "moe_debug_stall_gemms": (I, [I]),
        "moe_debug_lag_gemms": (I, [I]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def declared_symbols():
    """Names of the functions include/moe_gate.h declares."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"^[A-Za-z_][\w \*]*?\b(moe_\w+)\s*\(", text, re.M)))


def status_str(code) -> str:
    return load().moe_status_str(int(code)).decode()


def launch_count() -> int:
    return int(load().moe_launch_count())


def moe_debug_stall_gemms(n):
    """Error-path test hook: the next n tensor-core GEMM launches issue no
    operand copies, so each times out after about a second with
    MOE_ERR_TIMEOUT in its status word (n = 0 cancels)."""
    _check(load().moe_debug_stall_gemms(int(n)), "moe_debug_stall_gemms")


def moe_debug_lag_gemms(n):
    """Test hook: in the next n launches of the 4-bit products the copies of the
    second half of every row tile lag by 20 us a stage (n = 0 cancels)."""
    _check(load().moe_debug_lag_gemms(int(n)), "moe_debug_lag_gemms")


def _ptr(t, name="tensor", dtype=None, shape=None):
    """Device address of a contiguous CUDA tensor; checks the dtype and shape
    when given (a mismatch here would let a kernel read or write out of
    bounds).  None passes through as NULL.  A call of one small kernel spends
    most of its time here, so the checks are plain comparisons."""
    if t is None:
        return None
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype is not dtype and (type(dtype) is not tuple or t.dtype not in dtype):
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if not (t.is_cuda or _on_device(t)):
        raise ValueError(f"{name}: must be a CUDA tensor")
    return t.data_ptr()


def _on_device(t) -> bool:
    """What a tensor that is not CUDA's has to pass (a test's stand-in does)."""
    return t.is_cuda


def _i32():
    return torch.int32


def _f32():
    return torch.float32


def _dt(t):
    if t.dtype is torch.bfloat16:
        return MOE_BF16
    if t.dtype is torch.float32:
        return MOE_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


# The current stream's handle by device index.  Not one of torch's documented
# calls, so it may be missing; the documented way makes a Stream object first (2.9
# us against 0.3, of a small call's 7).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    """The stream's handle; None: torch's current stream of the current device."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return (torch.cuda.current_stream() if stream is None else stream).cuda_stream


def _check(code, where):
    if code != MOE_OK:
        raise MoEError(code, where)


def _act(act):
    return ACT[act] if isinstance(act, str) else int(act)


def _code(table, v, name):
    if isinstance(v, str):
        if v not in table:
            raise ValueError(f"{name}: {v!r}, expected one of {sorted(table)}")
        return table[v]
    return int(v)


# ------------------------------------------------------------------ sizes
def moe_capacity_bound(capacity_factor, s, e, k) -> int:
    return int(load().moe_capacity_bound(float(capacity_factor), int(s), int(e), int(k)))


def moe_capacity_workspace_size(s, e, k) -> int:
    return int(load().moe_capacity_workspace_size(int(s), int(e), int(k)))


def moe_expert_ffn_workspace_size(dtype, act, e, c_max, m, h) -> int:
    return int(load().moe_expert_ffn_workspace_size(int(dtype), _act(act), int(e), int(c_max),
                                                    int(m), int(h)))


def moe_expert_ffn_bwd_workspace_size(dtype, act, e, c_max, m, h) -> int:
    return int(load().moe_expert_ffn_bwd_workspace_size(int(dtype), _act(act), int(e), int(c_max),
                                                        int(m), int(h)))


def moe_layer_workspace_size(dtype, act, s, m, e, k, c_max, h) -> int:
    return int(load().moe_layer_workspace_size(int(dtype), _act(act), int(s), int(m), int(e),
                                               int(k), int(c_max), int(h)))


# ------------------------------------------------------------ entry points
def moe_gate_topk(x, wg, bias, k, idx, gates, dev_status, flags=0, stream=None):
    """x [s, m]; wg [m, e] fp32; bias [e] fp32 or None -> idx [k, s] int32, gates [k, s] fp32."""
    s, m = x.shape
    e = wg.shape[1]
    k = int(k)
    I, F = _i32(), _f32()
    _check(load().moe_gate_topk(
        _ptr(x, "x"), _dt(x), _ptr(wg, "wg", F, (m, e)), _ptr(bias, "bias", F, (e,)), s, m, e, k,
        int(flags), _ptr(idx, "idx", I, (k, s)), _ptr(gates, "gates", F, (k, s)),
        _ptr(dev_status, "dev_status", I), _stream(stream)), "moe_gate_topk")


def moe_capacity_locations(idx, e, capacity_factor, c_max, workspace, loc, counts, c_dev,
                           dev_status, stream=None):
    k, s = idx.shape
    I = _i32()
    _check(load().moe_capacity_locations(
        _ptr(idx, "idx", I), s, int(e), k, float(capacity_factor), int(c_max),
        _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _ptr(loc, "loc", I, (k, s)), _ptr(counts, "counts", I, (int(e),)),
        _ptr(c_dev, "c_dev", I), _ptr(dev_status, "dev_status", I), _stream(stream)),
        "moe_capacity_locations")


def moe_capacity_locations_noalloc(idx, e, capacity_factor, c_max, loc, counts, c_dev,
                                   dev_status, stream=None):
    """moe_capacity_locations with its scratch in the library's fixed device
    array (for callers that cannot allocate device memory); see the header."""
    k, s = idx.shape
    I = _i32()
    _check(load().moe_capacity_locations_noalloc(
        _ptr(idx, "idx", I), s, int(e), k, float(capacity_factor), int(c_max),
        _ptr(loc, "loc", I, (k, s)), _ptr(counts, "counts", I, (int(e),)),
        _ptr(c_dev, "c_dev", I), _ptr(dev_status, "dev_status", I), _stream(stream)),
        "moe_capacity_locations_noalloc")


def moe_encode(x, idx, loc, counts, c_dev, buf, dev_status, flags=0, stream=None):
    """buf is [e, c_max, m]."""
    s, m = x.shape
    k = idx.shape[0]
    e, c_max, _ = buf.shape
    I = _i32()
    _check(load().moe_encode(
        _ptr(x, "x"), _dt(x), _ptr(idx, "idx", I, (k, s)), _ptr(loc, "loc", I, (k, s)),
        _ptr(counts, "counts", I, (e,)), _ptr(c_dev, "c_dev", I), s, m, e, k, c_max, int(flags),
        _ptr(buf, "buf", x.dtype, (e, c_max, m)), _ptr(dev_status, "dev_status", I),
        _stream(stream)), "moe_encode")


def moe_expert_ffn(buf, counts, c_dev, w1, b1, w3, w2, b2, act, workspace, out, dev_status,
                   stream=None):
    e, c_max, m = buf.shape
    h = w1.shape[1]
    I, dt = _i32(), buf.dtype
    _check(load().moe_expert_ffn(
        _ptr(buf, "buf"), _dt(buf), _ptr(counts, "counts", I, (e,)), _ptr(c_dev, "c_dev", I),
        _ptr(w1, "w1", dt, (e, h, m)), _ptr(b1, "b1", dt, (e, h)), _ptr(w3, "w3", dt, (e, h, m)),
        _ptr(w2, "w2", dt, (e, m, h)), _ptr(b2, "b2", dt, (e, m)), _act(act), e, c_max, m, h,
        _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _ptr(out, "out", dt, (e, c_max, m)), _ptr(dev_status, "dev_status", I),
        _stream(stream)), "moe_expert_ffn")


def moe_expert_ffn_train(buf, counts, c_dev, w1, b1, w3, w2, b2, act, workspace, out, pre,
                         dev_status, stream=None):
    """moe_expert_ffn (bf16) that also keeps what moe_expert_ffn_bwd_saved
    needs: the pre-activation [e, c_max, h] (ReLU / GELU) or [a | b]
    [e, c_max, 2h] (SwiGLU)."""
    e, c_max, m = buf.shape
    h = w1.shape[1]
    I, dt = _i32(), buf.dtype
    hp = 2 * h if _act(act) == ACT["swiglu"] else h
    _check(load().moe_expert_ffn_train(
        _ptr(buf, "buf"), _dt(buf), _ptr(counts, "counts", I, (e,)), _ptr(c_dev, "c_dev", I),
        _ptr(w1, "w1", dt, (e, h, m)), _ptr(b1, "b1", dt, (e, h)), _ptr(w3, "w3", dt, (e, h, m)),
        _ptr(w2, "w2", dt, (e, m, h)), _ptr(b2, "b2", dt, (e, m)), _act(act), e, c_max, m, h,
        _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _ptr(out, "out", dt, (e, c_max, m)), _ptr(pre, "pre", dt, (e, c_max, hp)),
        _ptr(dev_status, "dev_status", I), _stream(stream)), "moe_expert_ffn_train")


def moe_expert_ffn_fp8_workspace_size(e, c_max, m, h) -> int:
    return int(load().moe_expert_ffn_fp8_workspace_size(int(e), int(c_max), int(m), int(h)))


def moe_quantize_rows_fp8(src, q, scale, dev_status, counts=None, c_dev=None, stream=None):
    """e4m3 codes (uint8, src's shape) and per-row fp32 scales of a bf16 tensor
    [rows, cols] or [batches, rows, cols]; with counts / c_dev only the kept
    rows of each batch."""
    shape = tuple(src.shape) if src.dim() == 3 else (1,) + tuple(src.shape)
    b, r, c = shape
    I = _i32()
    _check(load().moe_quantize_rows_fp8(
        _ptr(src, "src", torch.bfloat16), b, r, c,
        _ptr(counts, "counts", I, (b,)) if counts is not None else None,
        _ptr(c_dev, "c_dev", I) if c_dev is not None else None,
        _ptr(q, "q", torch.uint8, tuple(src.shape)),
        _ptr(scale, "scale", _f32(), tuple(src.shape[:-1])), _ptr(dev_status, "dev_status", I),
        _stream(stream)), "moe_quantize_rows_fp8")


def moe_expert_ffn_fp8(buf_q, buf_scale, counts, c_dev, w1_q, w1_scale, b1, w2_q, w2_scale, b2,
                       act, workspace, out, dev_status, stream=None):
    e, c_max, m = buf_q.shape
    h = w1_q.shape[1]
    I, F, U8, bf = _i32(), _f32(), torch.uint8, torch.bfloat16
    _check(load().moe_expert_ffn_fp8(
        _ptr(buf_q, "buf_q", U8), _ptr(buf_scale, "buf_scale", F, (e, c_max)),
        _ptr(counts, "counts", I, (e,)), _ptr(c_dev, "c_dev", I),
        _ptr(w1_q, "w1_q", U8, (e, h, m)), _ptr(w1_scale, "w1_scale", F, (e, h)),
        _ptr(b1, "b1", bf, (e, h)), _ptr(w2_q, "w2_q", U8, (e, m, h)),
        _ptr(w2_scale, "w2_scale", F, (e, m)), _ptr(b2, "b2", bf, (e, m)), _act(act), e, c_max,
        m, h, _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _ptr(out, "out", bf, (e, c_max, m)), _ptr(dev_status, "dev_status", I), _stream(stream)),
        "moe_expert_ffn_fp8")


# ------------------------------------------------------- routing from logits
def moe_route_topk(logits, bias, k, idx, gates, dev_status, score="softmax", groups=1,
                   topk_groups=1, group_top=1, scale=1.0, flags=0, stream=None):
    """logits [s, e] fp32 or bf16; bias [e] fp32 or None (steers the choice
    only) -> idx [k, s] int32, gates [k, s] fp32.  score "softmax" or
    "sigmoid"; the experts of the topk_groups best of `groups` runs compete, a
    group ranked by the sum of its group_top best; MOE_FLAG_NORMALIZE_GATES
    divides the gates by their sum, then `scale` multiplies them."""
    s, e = logits.shape
    k = int(k)
    I, F = _i32(), _f32()
    _check(load().moe_route_topk(
        _ptr(logits, "logits"), _dt(logits), _ptr(bias, "bias", F, (e,)), s, e, k,
        _code(SCORE, score, "score"), int(groups), int(topk_groups), int(group_top), float(scale),
        int(flags), _ptr(idx, "idx", I, (k, s)), _ptr(gates, "gates", F, (k, s)),
        _ptr(dev_status, "dev_status", I), _stream(stream)), "moe_route_topk")


def moe_route_bwd(logits, idx, d_gates, d_logits, dev_status, score="softmax", scale=1.0, flags=0,
                  stream=None):
    """Gradient of moe_route_topk's gates: d_gates [k, s] fp32 -> d_logits
    [s, e] (fp32 or bf16); score, scale and flags as given to the forward."""
    s, e = logits.shape
    k = idx.shape[0]
    I, F = _i32(), _f32()
    _check(load().moe_route_bwd(
        _ptr(logits, "logits"), _dt(logits), _ptr(idx, "idx", I, (k, s)),
        _ptr(d_gates, "d_gates", F, (k, s)), s, e, k, _code(SCORE, score, "score"), float(scale),
        int(flags), _ptr(d_logits, "d_logits", None, (s, e)), _dt(d_logits),
        _ptr(dev_status, "dev_status", I), _stream(stream)), "moe_route_bwd")


# ------------------------------------------------- microscaled 4-bit operands
def moe_fp4_scale_bytes(fmt, rows, cols) -> int:
    """Bytes of one batch's tiled block scales (0: cols not a multiple of 32)."""
    fmt = _code(FP4, fmt, "fmt")
    if fmt not in (0, 1) or rows < 1 or rows > 0x7FFFFFFF or cols < 32 or cols % 32:
        return 0
    return -(-rows // 128) * -(-cols // (128 if fmt == 0 else 64)) * 512   # moe_fp4_scale_bytes of the C ABI


def _fp4(q, scale, fmt, name, batches, rows, cols):
    """Addresses of a 4-bit operand's codes and scales (fmt: the format's code)."""
    n = -(-rows // 128) * -(-cols // (128 if fmt == 0 else 64)) * 512   # moe_fp4_scale_bytes
    return (_ptr(q, name, torch.uint8, (batches, rows, cols // 2)),
            _ptr(scale, name[:-1] + "scale", torch.uint8, (batches, n)))


def _batched(t):
    return tuple(t.shape) if t.dim() == 3 else (1,) + tuple(t.shape)


def moe_quantize_fp4(src, fmt, q, scale, dev_status, global_scale=None, counts=None, c_dev=None,
                     stream=None):
    """4-bit codes (uint8 [..., cols/2], two a byte) and tiled block scales
    (uint8 [batches, moe_fp4_scale_bytes]) of src [rows, cols] or [batches,
    rows, cols] (bf16 or fp32); fmt "mx" or "nv", the latter with a factor per
    batch (global_scale [batches] fp32, None: 1); with counts / c_dev only the
    kept rows of each batch."""
    b, r, c = _batched(src)
    I, fmt = _i32(), _code(FP4, fmt, "fmt")
    qp, sp = _fp4(q if src.dim() == 3 else q.unsqueeze(0), scale, fmt, "q", b, r, c)
    _check(load().moe_quantize_fp4(
        _ptr(src, "src"), _dt(src), b, r, c, fmt,
        _ptr(global_scale, "global_scale", _f32(), (b,)), _ptr(counts, "counts", I, (b,)),
        _ptr(c_dev, "c_dev", I), qp, sp, _ptr(dev_status, "dev_status", I), _stream(stream)),
        "moe_quantize_fp4")


def moe_dequantize_fp4(q, scale, fmt, dst, dev_status, global_scale=None, counts=None, c_dev=None,
                       stream=None):
    """The values of moe_quantize_fp4's codes and scales, into dst [rows, cols]
    or [batches, rows, cols] (bf16 or fp32)."""
    b, r, c = _batched(dst)
    I, fmt = _i32(), _code(FP4, fmt, "fmt")
    qp, sp = _fp4(q if dst.dim() == 3 else q.unsqueeze(0), scale, fmt, "q", b, r, c)
    _check(load().moe_dequantize_fp4(
        qp, sp, b, r, c, fmt, _ptr(global_scale, "global_scale", _f32(), (b,)),
        _ptr(counts, "counts", I, (b,)), _ptr(c_dev, "c_dev", I), _ptr(dst, "dst"), _dt(dst),
        _ptr(dev_status, "dev_status", I), _stream(stream)), "moe_dequantize_fp4")


def moe_product_fp4(a_q, a_scale, a_global, counts, c_dev, b_q, b_scale, b_global, bias, fmt, out,
                    dev_status, stream=None):
    """out[j] = a[j] b[j]^T (+ bias[j]) over the kept rows of every expert:
    a_q [e, c_max, k/2], b_q [e, n, k/2] with their scales and factors ([e] fp32
    or None), bias [e, n] bf16 or None, out [e, c_max, n] bf16."""
    e, c_max, n = out.shape
    k = 2 * a_q.shape[2]
    I, F, bf, fmt = _i32(), _f32(), torch.bfloat16, _code(FP4, fmt, "fmt")
    ap, asp = _fp4(a_q, a_scale, fmt, "a_q", e, c_max, k)
    bp, bsp = _fp4(b_q, b_scale, fmt, "b_q", e, n, k)
    _check(load().moe_product_fp4(
        ap, asp, _ptr(a_global, "a_global", F, (e,)), _ptr(counts, "counts", I, (e,)),
        _ptr(c_dev, "c_dev", I), bp, bsp, _ptr(b_global, "b_global", F, (e,)),
        _ptr(bias, "bias", bf, (e, n)), fmt, e, c_max, k, n,
        _ptr(out, "out", bf), _ptr(dev_status, "dev_status", I), _stream(stream)),
        "moe_product_fp4")


def moe_expert_ffn_fp4_workspace_size(fmt, act, e, c_max, m, h) -> int:
    return int(load().moe_expert_ffn_fp4_workspace_size(_code(FP4, fmt, "fmt"), _act(act), int(e),
                                                        int(c_max), int(m), int(h)))


def moe_expert_ffn_fp4(buf_q, buf_scale, buf_global, hid_global, counts, c_dev, w1_q, w1_scale,
                       w1_global, b1, w3_q, w3_scale, w3_global, w2_q, w2_scale, w2_global, b2, fmt,
                       act, workspace, out, dev_status, stream=None):
    """The expert FFN on 4-bit operands (moe_quantize_fp4 of the buffer's kept
    rows and of the weights [e, h, m], [e, h, m], [e, m, h]); factors [e] fp32
    or None; w3 and its scales only for SwiGLU, which takes no biases."""
    e, c_max, m = out.shape
    h = w1_q.shape[1]
    I, F, bf, fmt = _i32(), _f32(), torch.bfloat16, _code(FP4, fmt, "fmt")
    xp, xsp = _fp4(buf_q, buf_scale, fmt, "buf_q", e, c_max, m)
    w1p, w1sp = _fp4(w1_q, w1_scale, fmt, "w1_q", e, h, m)
    w3p, w3sp = _fp4(w3_q, w3_scale, fmt, "w3_q", e, h, m)
    w2p, w2sp = _fp4(w2_q, w2_scale, fmt, "w2_q", e, m, h)
    _check(load().moe_expert_ffn_fp4(
        xp, xsp, _ptr(buf_global, "buf_global", F, (e,)), _ptr(hid_global, "hid_global", F, (e,)),
        _ptr(counts, "counts", I, (e,)), _ptr(c_dev, "c_dev", I), w1p, w1sp,
        _ptr(w1_global, "w1_global", F, (e,)), _ptr(b1, "b1", bf, (e, h)), w3p, w3sp,
        _ptr(w3_global, "w3_global", F, (e,)), w2p, w2sp, _ptr(w2_global, "w2_global", F, (e,)),
        _ptr(b2, "b2", bf, (e, m)), fmt, _act(act), e, c_max, m, h,
        _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _ptr(out, "out", bf), _ptr(dev_status, "dev_status", I), _stream(stream)),
        "moe_expert_ffn_fp4")


def moe_expert_ffn_bwd(buf, hid, counts, c_dev, w1, b1, w3, w2, act, d_out, workspace, d_buf,
                       d_w1, d_w3, d_w2, d_b1, d_b2, dev_status, stream=None):
    """Gradient of moe_expert_ffn over the kept rows (bf16); hid is the
    forward's hidden (its workspace after the call)."""
    e, c_max, m = buf.shape
    h = w1.shape[1]
    I, dt = _i32(), buf.dtype
    _check(load().moe_expert_ffn_bwd(
        _ptr(buf, "buf"), _ptr(hid, "hid", dt, (e, c_max, h)), _dt(buf),
        _ptr(counts, "counts", I, (e,)), _ptr(c_dev, "c_dev", I), _ptr(w1, "w1", dt, (e, h, m)),
        _ptr(b1, "b1", dt, (e, h)), _ptr(w3, "w3", dt, (e, h, m)), _ptr(w2, "w2", dt, (e, m, h)),
        _act(act), e, c_max, m, h, _ptr(d_out, "d_out", dt, (e, c_max, m)),
        _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _ptr(d_buf, "d_buf", dt, (e, c_max, m)), _ptr(d_w1, "d_w1", dt, (e, h, m)),
        _ptr(d_w3, "d_w3", dt, (e, h, m)), _ptr(d_w2, "d_w2", dt, (e, m, h)),
        _ptr(d_b1, "d_b1", dt, (e, h)), _ptr(d_b2, "d_b2", dt, (e, m)),
        _ptr(dev_status, "dev_status", I), _stream(stream)), "moe_expert_ffn_bwd")


def moe_expert_ffn_bwd_saved(buf, hid, pre, counts, c_dev, w1, w3, w2, act, d_out, workspace,
                             d_buf, d_w1, d_w3, d_w2, d_b1, d_b2, dev_status, stream=None):
    """moe_expert_ffn_bwd with what moe_expert_ffn_train kept: nothing is
    recomputed.  The weight and bias gradients are all bf16 or all fp32
    (kept in fp32); w3 / d_w3 for SwiGLU only."""
    e, c_max, m = buf.shape
    h = w1.shape[1]
    I, dt = _i32(), buf.dtype
    hp = 2 * h if _act(act) == ACT["swiglu"] else h
    gdt = d_w1.dtype
    if gdt not in (torch.bfloat16, torch.float32):
        raise ValueError(f"d_w1: dtype {gdt}, expected bfloat16 or float32")
    _check(load().moe_expert_ffn_bwd_saved(
        _ptr(buf, "buf"), _ptr(hid, "hid", dt, (e, c_max, h)),
        _ptr(pre, "pre", dt, (e, c_max, hp)), _dt(buf), _ptr(counts, "counts", I, (e,)),
        _ptr(c_dev, "c_dev", I), _ptr(w1, "w1", dt, (e, h, m)), _ptr(w3, "w3", dt, (e, h, m)),
        _ptr(w2, "w2", dt, (e, m, h)), _act(act), e, c_max, m, h,
        _ptr(d_out, "d_out", dt, (e, c_max, m)),
        _ptr(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _ptr(d_buf, "d_buf", dt, (e, c_max, m)), _dt(d_w1), _ptr(d_w1, "d_w1", gdt, (e, h, m)),
        _ptr(d_w3, "d_w3", gdt, (e, h, m)),
        _ptr(d_w2, "d_w2", gdt, (e, m, h)), _ptr(d_b1, "d_b1", gdt, (e, h)),
        _ptr(d_b2, "d_b2", gdt, (e, m)), _ptr(dev_status, "dev_status", I), _stream(stream)),
        "moe_expert_ffn_bwd_saved")


def moe_decode(out, idx, loc, gates, c_dev, y, dev_status, stream=None):
    e, c_max, m = out.shape
    k, s = idx.shape
    I, F = _i32(), _f32()
    _check(load().moe_decode(
        _ptr(out, "out"), _dt(out), _ptr(idx, "idx", I), _ptr(loc, "loc", I, (k, s)),
        _ptr(gates, "gates", F, (k, s)), _ptr(c_dev, "c_dev", I), s, m, e, k, c_max,
        _ptr(y, "y", out.dtype, (s, m)), _ptr(dev_status, "dev_status", I), _stream(stream)),
        "moe_decode")


def moe_decode_bwd(dy, out, idx, loc, gates, counts, c_dev, d_out, d_gates, dev_status, flags=0,
                   stream=None):
    e, c_max, m = out.shape
    k, s = idx.shape
    I, F, dt = _i32(), _f32(), out.dtype
    _check(load().moe_decode_bwd(
        _ptr(dy, "dy", dt, (s, m)), _ptr(out, "out"), _dt(out), _ptr(idx, "idx", I),
        _ptr(loc, "loc", I, (k, s)), _ptr(gates, "gates", F, (k, s)),
        _ptr(counts, "counts", I, (e,)), _ptr(c_dev, "c_dev", I), s, m, e, k, c_max, int(flags),
        _ptr(d_out, "d_out", dt, (e, c_max, m)), _ptr(d_gates, "d_gates", F, (k, s)),
        _ptr(dev_status, "dev_status", I), _stream(stream)), "moe_decode_bwd")


def moe_gate_bwd(x, wg, bias, idx, gates, d_gates, d_logits, dev_status, d_wg=None, d_bias=None,
                 d_x=None, flags=0, stream=None):
    """Gate backward: d_gates [k, s] fp32 -> d_logits [s, e] and, when given,
    d_wg [m, e], d_bias [e], d_x [s, m] (all fp32)."""
    s, m = x.shape
    e = wg.shape[1]
    k = idx.shape[0]
    I, F = _i32(), _f32()
    _check(load().moe_gate_bwd(
        _ptr(x, "x"), _dt(x), _ptr(wg, "wg", F, (m, e)), _ptr(bias, "bias", F, (e,)), s, m, e, k,
        int(flags), _ptr(idx, "idx", I, (k, s)), _ptr(gates, "gates", F, (k, s)),
        _ptr(d_gates, "d_gates", F, (k, s)), _ptr(d_logits, "d_logits", F, (s, e)),
        _ptr(d_wg, "d_wg", F, (m, e)), _ptr(d_bias, "d_bias", F, (e,)),
        _ptr(d_x, "d_x", F, (s, m)), _ptr(dev_status, "dev_status", I), _stream(stream)),
        "moe_gate_bwd")


def moe_encode_bwd(d_buf, idx, loc, c_dev, dx, dev_status, stream=None):
    e, c_max, m = d_buf.shape
    k, s = idx.shape
    I = _i32()
    _check(load().moe_encode_bwd(
        _ptr(d_buf, "d_buf"), _dt(d_buf), _ptr(idx, "idx", I), _ptr(loc, "loc", I, (k, s)),
        _ptr(c_dev, "c_dev", I), s, m, e, k, c_max, _ptr(dx, "dx", d_buf.dtype, (s, m)),
        _ptr(dev_status, "dev_status", I), _stream(stream)), "moe_encode_bwd")


def moe_layer_forward(x, wg, gate_bias, w1, b1, w3, w2, b2, act, k, capacity_factor, flags,
                      idx, gates, loc, counts, c_dev, buf, out, y, workspace, dev_status,
                      stream=None):
    s, m = x.shape
    e, c_max, _ = buf.shape
    h = w1.shape[1]
    k = int(k)
    I, F, dt = _i32(), _f32(), x.dtype
    _check(load().moe_layer_forward(
        _ptr(x, "x"), _dt(x), _ptr(wg, "wg", F, (m, e)), _ptr(gate_bias, "gate_bias", F, (e,)),
        _ptr(w1, "w1", dt, (e, h, m)), _ptr(b1, "b1", dt, (e, h)), _ptr(w3, "w3", dt, (e, h, m)),
        _ptr(w2, "w2", dt, (e, m, h)), _ptr(b2, "b2", dt, (e, m)), _act(act), s, m, e, k, h,
        float(capacity_factor), c_max, int(flags), _ptr(idx, "idx", I, (k, s)),
        _ptr(gates, "gates", F, (k, s)), _ptr(loc, "loc", I, (k, s)),
        _ptr(counts, "counts", I, (e,)), _ptr(c_dev, "c_dev", I), _ptr(buf, "buf", dt, (e, c_max, m)),
        _ptr(out, "out", dt, (e, c_max, m)), _ptr(y, "y", dt, (s, m)), _ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _ptr(dev_status, "dev_status", I),
        _stream(stream)), "moe_layer_forward")


def moe_layer_forward_host(x_host, y_host, x, wg, gate_bias, w1, b1, w3, w2, b2, act, k,
                           capacity_factor, flags, idx, gates, loc, counts, c_dev, buf, out, y,
                           workspace, dev_status, stream=None):
    """moe_layer_forward with x read from, and y written to, host tensors
    (pinned for asynchronous copies); x and y are the device buffers."""
    s, m = x.shape
    e, c_max, _ = buf.shape
    h = w1.shape[1]
    k = int(k)
    I, F, dt = _i32(), _f32(), x.dtype
    for name, t in (("x_host", x_host), ("y_host", y_host)):
        if t.is_cuda or tuple(t.shape) != (s, m) or t.dtype != dt or not t.is_contiguous():
            raise ValueError(f"{name}: must be a contiguous host tensor [{s}, {m}] of {dt}")
    _check(load().moe_layer_forward_host(
        ctypes.c_void_p(x_host.data_ptr()), ctypes.c_void_p(y_host.data_ptr()), _ptr(x, "x"), _dt(x),
        _ptr(wg, "wg", F, (m, e)), _ptr(gate_bias, "gate_bias", F, (e,)),
        _ptr(w1, "w1", dt, (e, h, m)), _ptr(b1, "b1", dt, (e, h)), _ptr(w3, "w3", dt, (e, h, m)),
        _ptr(w2, "w2", dt, (e, m, h)), _ptr(b2, "b2", dt, (e, m)), _act(act), s, m, e, k, h,
        float(capacity_factor), c_max, int(flags), _ptr(idx, "idx", I, (k, s)),
        _ptr(gates, "gates", F, (k, s)), _ptr(loc, "loc", I, (k, s)),
        _ptr(counts, "counts", I, (e,)), _ptr(c_dev, "c_dev", I), _ptr(buf, "buf", dt, (e, c_max, m)),
        _ptr(out, "out", dt, (e, c_max, m)), _ptr(y, "y", dt, (s, m)), _ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _ptr(dev_status, "dev_status", I),
        _stream(stream)), "moe_layer_forward_host")


def moe_layer_forward_pipelined(x, wg, gate_bias, w1, b1, w3, w2, b2, act, k, capacity_factor,
                                flags, idx, gates, loc, counts, c_dev, buf, out, y, workspace,
                                dev_status, chunks, aux_stream, events, stream=None):
    """moe_layer_forward with encode of capacity chunk i+1 (on aux_stream)
    overlapping the FFN of chunk i (on stream); events: 1 + chunks
    torch.cuda.Event objects."""
    s, m = x.shape
    e, c_max, _ = buf.shape
    h = w1.shape[1]
    k, chunks = int(k), int(chunks)
    if len(events) < chunks + 1:
        raise ValueError(f"events: need {chunks + 1}, got {len(events)}")
    for ev in events[:chunks + 1]:   # the handles exist once the events are recorded or created
        if getattr(ev, "cuda_event", 0) == 0:
            ev.record(torch_current_stream())
    handles = (ctypes.c_void_p * (chunks + 1))(*[ctypes.c_void_p(ev.cuda_event) for ev in
                                                 events[:chunks + 1]])
    I, F, dt = _i32(), _f32(), x.dtype
    _check(load().moe_layer_forward_pipelined(
        _ptr(x, "x"), _dt(x), _ptr(wg, "wg", F, (m, e)), _ptr(gate_bias, "gate_bias", F, (e,)),
        _ptr(w1, "w1", dt, (e, h, m)), _ptr(b1, "b1", dt, (e, h)), _ptr(w3, "w3", dt, (e, h, m)),
        _ptr(w2, "w2", dt, (e, m, h)), _ptr(b2, "b2", dt, (e, m)), _act(act), s, m, e, k, h,
        float(capacity_factor), c_max, int(flags), _ptr(idx, "idx", I, (k, s)),
        _ptr(gates, "gates", F, (k, s)), _ptr(loc, "loc", I, (k, s)),
        _ptr(counts, "counts", I, (e,)), _ptr(c_dev, "c_dev", I), _ptr(buf, "buf", dt, (e, c_max, m)),
        _ptr(out, "out", dt, (e, c_max, m)), _ptr(y, "y", dt, (s, m)), _ptr(workspace, "workspace"),
        workspace.numel() * workspace.element_size(), _ptr(dev_status, "dev_status", I), chunks,
        _stream(stream), _stream(aux_stream), handles), "moe_layer_forward_pipelined")


def torch_current_stream():
    return torch.cuda.current_stream()


def moe_probe_fp32_fma(packed, blocks, iters, out, stream=None):
    """Launch the fp32 FMA throughput probe (blocks * 256 * iters * 32 flop)."""
    _check(load().moe_probe_fp32_fma(int(bool(packed)), int(blocks), int(iters),
                                     _ptr(out, "out", _f32()), _stream(stream)), "moe_probe_fp32_fma")


from .layer import (Fp4Operand, MoELayerBuffers, MoELayerFp4Buffers, alloc_layer,  # noqa: E402,F401
                    alloc_layer_fp4, quantize_weights_fp4, run_layer, run_layer_fp4, run_layer_host)
