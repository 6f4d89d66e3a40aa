"""How the attention kernels share units among CTAs (csrc/work_split.h), compiled for the host."""
import ctypes
import os
import shutil
import subprocess

import pytest

from lfm2_gated_short_gb300 import build as sc_build


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    d = tmp_path_factory.mktemp("work_split")
    src, so = d / "s.cpp", d / "s.so"
    src.write_text('#include "work_split.h"\n'
                   'extern "C" int64_t begin(int64_t c, int64_t U, int64_t n)'
                   ' { return sc::share_begin(c, U, n); }\n'
                   'extern "C" int of(int64_t u, int64_t U, int64_t n) { return sc::share_of(u, U, n); }\n')
    cxx = shutil.which("g++") or shutil.which("c++")
    subprocess.run([cxx, "-O1", "-std=c++17", "-shared", "-fPIC", "-I", sc_build.CSRC, os.fspath(src),
                    "-o", os.fspath(so)], check=True)
    lib = ctypes.CDLL(os.fspath(so))
    lib.begin.argtypes, lib.begin.restype = [ctypes.c_int64] * 3, ctypes.c_int64
    lib.of.argtypes, lib.of.restype = [ctypes.c_int64] * 3, ctypes.c_int
    return lib


@pytest.mark.parametrize("U", [1, 2, 7, 456, 457, 10 ** 6, 2 ** 32 // 456, 2 ** 32 // 456 + 1,
                               2 ** 32 - 1, 2 ** 32, 2 ** 32 + 1, 3 * 2 ** 32 + 5, 2 ** 40])
@pytest.mark.parametrize("n", [1, 2, 3, 32, 152, 455, 456])
def test_every_unit_belongs_to_the_cta_whose_share_holds_it(L, U, n):
    n = min(n, U)
    assert L.begin(0, U, n) == 0 and L.begin(n, U, n) == U
    for c in range(n):
        b, e = L.begin(c, U, n), L.begin(c + 1, U, n)
        assert b == c * U // n and b < e
        for u in {b, b + 1, (b + e) // 2, e - 1}:
            if b <= u < e:
                assert L.of(u, U, n) == c, (u, c)
