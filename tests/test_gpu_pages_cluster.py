"""The paged cache where a cluster of CTAs works a call out and the lanes of a warp differ: listed
sequences that grow, shrink, are copied, do not change or are skipped, side by side."""
import numpy as np
import pytest

from test_gpu_pages import Pair

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [300, 1100])
def test_mixed_lanes(n):
    r = np.random.default_rng(n)
    ps, max_pages = 8, 20
    p = Pair(n + 5, max_pages, 12 * n, ps, Hkv=1, Dh=8, seed=n)
    p.resize([0, 1], [ps * 11 + 3, ps * 6])
    branches = np.arange(2, n + 2)
    p.fork(r.integers(0, 2, n), branches)
    for _ in range(3):
        slots = r.permutation(branches)
        slots[r.random(n) < 0.1] = -1                       # skipped
        slots[r.random(n) < 0.1] = n + 5 + 7
        now = np.where(slots < n + 5, p.m.lens[np.clip(slots, 0, n + 4)], 0)
        new = now + r.integers(-30, 20, n) * (r.random(n) < 0.8)
        new = np.where(r.random(n) < 0.1, 0, np.maximum(new, 0))
        new[r.random(n) < 0.05] = ps * max_pages + 1        # skipped
        p.resize(slots, new)
        dst = r.permutation(branches)[:n // 2]
        src = np.where(r.random(n // 2) < 0.5, 0, 1)
        src[r.random(n // 2) < 0.2] = -3                    # skipped
        p.fork(src, dst)
    p.compact()
