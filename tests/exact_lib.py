"""Builds and loads tests/cuda/exact.cu, once per test session."""

import ctypes
import functools
import os
import subprocess
import tempfile

import torch

from combine_moe_gate_gb300 import build as B

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "cuda", "exact.cu")


@functools.lru_cache(None)
def load():
    out = os.path.join(tempfile.mkdtemp(prefix="exact_"), "libexact.so")
    subprocess.run([B._nvcc(), *B._flags(False), "-shared", "-o", out, SRC], check=True, capture_output=True)
    lib = ctypes.CDLL(out)
    P, I, U = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint32
    lib.exact_rcp.argtypes = [U, U, P]
    lib.exact_div.argtypes = [U, I, I, I, I, I, I, P]
    lib.exact_exp.argtypes = [P, P, ctypes.c_int64]
    return lib


def expf(x):
    """CUDA's expf of an fp32 tensor."""
    x = x.contiguous()
    y = torch.empty_like(x)
    torch.cuda.synchronize()
    assert load().exact_exp(x.data_ptr(), y.data_ptr(), x.numel()) == 0
    torch.cuda.synchronize()
    return y
