"""prefix_attention where a share of the prefix's work runs from items of two row tiles into items of
one: an odd number of row tiles, more than one, and fewer CTAs than items. Bound as in
test_gpu_prefix_attention.py."""
import pytest
import torch

from test_gpu_prefix_attention import build, call, check

pytestmark = pytest.mark.gpu


# Row tiles hold 128 / G tokens. With 8 units a CTA (4 with heads of 128), a unit a 128-key tile, items
# of 3 or 5 units end inside a CTA's share; the items of one row tile come last.
@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("Hkv,G,N,D", [(3, 4, 65, 1), (4, 4, 22, 4), (3, 32, 17, 1), (5, 7, 40, 1)])
@pytest.mark.parametrize("keys", [300, 640])
def test_two_row_tiles_then_one(Dh, Hkv, G, N, D, keys):
    tiles = -(-N * D // (128 // G))
    assert tiles % 2 == 1 and tiles > 1
    shared = keys // 8
    c = build([shared * 8 + D + i % 5 for i in range(N)], shared=shared, ps=8, D=D, Hkv=Hkv, G=G, Dh=Dh,
              seed=N)
    check(c)
    first = call(c)
    for _ in range(20):
        assert torch.equal(call(c), first)
