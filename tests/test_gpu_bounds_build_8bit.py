"""The 8-bit cache's and the rotary operators' guard-band file under the bounds-checked build (see
test_gpu_bounds_build.py): every refused access fails its tests, and those that shorten a
record see the kernels' own accesses refused."""
import os
import subprocess
import sys

import pytest

from lfm2_gated_short_gb300 import build as sc_build

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


def test_8bit_guard_band_cases_under_the_bounds_checked_build():
    lib = sc_build.build(bounds_check=True)
    env = dict(os.environ, SHORTCONV_LIBRARY=lib)
    r = subprocess.run(
        [sys.executable, "-m", "pytest", os.path.join(HERE, "test_gpu_guard_bands_8bit.py"), "-m",
         "gpu", "-q", "-rs", "-p", "no:cacheprovider"],
        cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    tail = (r.stdout + r.stderr)[-4000:]
    assert r.returncode == 0, tail
    assert " passed" in r.stdout and "skipped" not in r.stdout, tail
