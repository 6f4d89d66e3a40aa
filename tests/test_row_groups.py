"""How reading the 8-bit cache back counts its groups of rows (csrc/work_split.h), compiled for the
host: a call may have 2^31 - 1 rows, and rounding up must not pass 32 bits."""
import ctypes
import os
import shutil
import subprocess

import pytest

from lfm2_gated_short_gb300 import build as sc_build


@pytest.fixture(scope="module")
def groups(tmp_path_factory):
    d = tmp_path_factory.mktemp("row_groups")
    src, so = d / "s.cpp", d / "s.so"
    src.write_text('#include "work_split.h"\n'
                   'extern "C" int64_t groups(int rows, int R) { return sc::row_groups(rows, R); }\n')
    cxx = shutil.which("g++") or shutil.which("c++")
    subprocess.run([cxx, "-O1", "-std=c++17", "-shared", "-fPIC", "-I", sc_build.CSRC, os.fspath(src),
                    "-o", os.fspath(so)], check=True)
    f = ctypes.CDLL(os.fspath(so)).groups
    f.argtypes, f.restype = [ctypes.c_int] * 2, ctypes.c_int64
    return f


@pytest.mark.parametrize("rows", [0, 1, 2, 31, 32, 33, 1000, 2 ** 31 - 33, 2 ** 31 - 2, 2 ** 31 - 1])
@pytest.mark.parametrize("R", [1, 2, 3, 21, 32])
def test_groups_hold_every_row(groups, rows, R):
    assert groups(rows, R) == -(-rows // R)
