"""Attention over the 8-bit cache behind tiles that never arrive: the waits run out (about 2 s each
call), DEV_TIMEOUT is set, no row is written, and the next call is right. The bounds-checked build
holds the tiles back, on the host's word; nothing faults."""
import os
import subprocess
import sys

import pytest
import torch

import lfm2_gated_short_gb300 as sc
from cache8_util import attend, build, on_device
from lfm2_gated_short_gb300 import build as sc_build

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


# One tile a CTA, so that every row's part is lost: items of one, two and four heads, of 8, 16 and 32
# rows, rows of one part and of several.
CASES = [(64, 1, 3, 1), (64, 2, 4, 2), (64, 4, 2, 1), (64, 1, 8, 4), (128, 1, 5, 2), (128, 4, 1, 3),
         (128, 2, 7, 3)]


def test_rows_whose_tiles_are_lost_are_left_alone():
    if not sc.bounds_checked():
        return  # the standard build holds no tile back
    for Dh, Hkv, G, D in CASES:
        c = build([9, 70, 300], Hkv=Hkv, G=G, D=D, Dh=Dh, seed=G)
        want = attend(c)
        d = on_device(c)
        out = torch.full(c["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        assert sc.get_error() == 0
        sc.bounds_starve_next()
        args = (d["q"], d["k"], d["v"], d["table"], d["lens"], d["slots"], D)
        sc.prefix_attention(*args, k_scales=d["ks"], v_scales=d["vs"], out=out)
        assert sc.get_error() == sc.DEV_TIMEOUT
        assert (out == 7.0).all()
        sc.prefix_attention(*args, k_scales=d["ks"], v_scales=d["vs"], out=out)
        assert sc.get_error() == 0
        assert torch.equal(out, want)


def test_lost_tiles_under_the_bounds_checked_build():
    if sc.bounds_checked():
        return  # the child process
    lib = sc_build.build(bounds_check=True)
    r = subprocess.run(
        [sys.executable, "-m", "pytest", os.path.abspath(__file__), "-m", "gpu", "-q", "-p",
         "no:cacheprovider"],
        cwd=ROOT, env=dict(os.environ, SHORTCONV_LIBRARY=lib), capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0 and " passed" in r.stdout, (r.stdout + r.stderr)[-4000:]


def test_the_standard_build_holds_no_tile_back():
    if not sc.bounds_checked():
        with pytest.raises(RuntimeError):
            sc.bounds_starve_next()
