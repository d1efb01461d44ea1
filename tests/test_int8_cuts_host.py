"""How the 8-bit grouped product cuts an expert's rows into tiles, on the host: the kernel's own function,
compiled by the host's compiler, over counts up to the largest buffer."""

import ctypes
import os
import random
import re
import subprocess

import pytest

import combine_moe_gate_gb300.build as B

NT, MAX_ROWS = 192, 2 ** 31 - 1024          # rows a tile at most; rows a buffer at most


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    with open(os.path.join(B.CSRC, "ffn_int8.cuh")) as f:
        body = re.search(r"int i8_cut\(int rows, int tiles\) \{.*?\}", f.read(), re.S).group(0)
    d = tmp_path_factory.mktemp("cuts")
    src, lib = d / "cut.cpp", d / "libcut.so"
    src.write_text(f'#include <cstdint>\nextern "C" {body}\n')
    # signed overflow wraps, as it does on the device
    subprocess.run(["g++", "-O1", "-fwrapv", "-shared", "-fPIC", "-o", str(lib), str(src)], check=True)
    fn = ctypes.CDLL(str(lib)).i8_cut
    fn.argtypes, fn.restype = [ctypes.c_int, ctypes.c_int], ctypes.c_int
    return fn


def test_every_row_is_in_one_tile(cut):
    rng = random.Random(5)
    counts = list(range(1, 1200)) + [MAX_ROWS - i for i in range(400)] + [2 ** 31 * 192 // 193 + i for i in range(-200, 200)]
    counts += [rng.randrange(1, MAX_ROWS + 1) for _ in range(2000)]
    for rows in counts:
        tiles = -(-rows // NT)
        per = cut(rows, tiles)
        assert 32 <= per <= NT and per % 32 == 0, (rows, per)
        assert (tiles - 1) * per < rows <= tiles * per, (rows, per)     # none empty, none left over
