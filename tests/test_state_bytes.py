"""CPU: the arithmetic of what the reordering of states moves, compiled for the host."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_verification_61_gb300", "csrc")


@pytest.fixture(scope="module")
def moved(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("state_bytes")
    (d / "m.cpp").write_text('#include "state_bytes.h"\nextern "C" int64_t moved(int64_t r, int64_t u, int32_t T, int32_t n) '
                             '{ return specstate::moved_bytes(r, u, T, n); }\n')
    subprocess.run(["g++", "-std=c++17", "-O2", "-fsanitize=undefined", "-fno-sanitize-recover", "-shared", "-fPIC", f"-I{CSRC}", "-o", str(d / "m.so"), str(d / "m.cpp")],
                   check=True)
    fn = ctypes.CDLL(str(d / "m.so")).moved
    fn.argtypes, fn.restype = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32], ctypes.c_int64
    return fn


ALL = 2 ** 31 - 1


@pytest.mark.parametrize("T,unit", [(1, 16), (1, 4 << 30), (1, (4 << 30) + 16), (1, 5 * 10 ** 9), (1, 13 * 10 ** 9), (1, 1 << 62), (2, (4 << 30) + 16), (3, 1 << 40),
                                    (7, 1), (ALL, 1), (ALL, 1 << 31), (ALL, 1 << 32)])
@pytest.mark.parametrize("length", [1, 2, 5, 1 << 16, ALL - 1, ALL])
def test_the_first_positions(moved, T, unit, length):
    assert moved(T * unit, unit, T, length) == min(T, length) * unit
