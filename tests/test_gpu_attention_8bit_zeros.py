"""Attention over the 8-bit cache where the blocks' V scales lie up to 2^184 apart, against float64:
blocks of zeros, whose scale is the least that there is, count in the sum that a row is divided by,
beside blocks of large values, inside a tile, a part and between parts. Bounds as in
test_gpu_attention_8bit_range.py."""
import numpy as np
import pytest
import torch

import lfm2_gated_short_gb300 as sc
from cache8_util import build, codes_from, i32
from test_gpu_attention_8bit_range import SHAPES, check

pytestmark = pytest.mark.gpu


def zeros_beside(c, up, zero):
    """V scales 2^up and random codes, but for the blocks that zero(block number of the sequence)
    names: codes of zero and the least scale."""
    ps, B = c["v"].shape[1], c["v"].shape[1] // c["vs"].shape[1]
    live = ~np.isnan(c["vs"])
    c["vs"][live] = np.float32(2.0 ** up)
    for s in c["slots"]:
        n = int(c["lens"][s])
        for b in range(-(-n // B)):
            page, e = c["table"][s, b * B // ps], b % (ps // B)
            if zero(b):
                rows = slice(e * B, min((e + 1) * B, ps))
                c["v"][page, rows][c["v"][page, rows] != 0x7F] = 0
                c["vs"][page, e] = np.float32(2.0 ** -64)
    return c


@pytest.mark.parametrize("up", [40, 62, 70, 100, 112])
@pytest.mark.parametrize("Dh,Hkv,G,D", SHAPES)
@pytest.mark.parametrize("every", [(0, 2), (1, 2), (0, 3), (2, 3)])
def test_zeros_beside_large_values(Dh, Hkv, G, D, up, every):
    at, of = every
    check(zeros_beside(build([300, 45, 9], D=D, G=G, Hkv=Hkv, Dh=Dh, B=8, seed=up), up,
                       lambda b: b % of == at), Dh ** -0.5)


@pytest.mark.parametrize("up", [62, 100])
@pytest.mark.parametrize("order", ["zeros first", "zeros last", "zeros between"])
@pytest.mark.parametrize("N,G,D", [(1, 4, 1), (9, 4, 8), (9, 8, 16)])
def test_parts_of_zeros_beside_parts_of_large_values(N, G, D, order, up):
    """Long sequences, in many parts, joined a block a row, a warp a row and eight lanes a row."""
    n = 9000 if N == 1 else 1500
    c = build([n - 31 * i for i in range(N)], Hkv=4, D=D, G=G, ps=64, B=64, seed=8)
    half = n // 128
    zero = {"zeros first": lambda b: b < half, "zeros last": lambda b: b >= half,
            "zeros between": lambda b: half // 2 < b < half * 3 // 2}[order]
    check(zeros_beside(c, up, zero), 0.125)


@pytest.mark.parametrize("up", [62, 90])
@pytest.mark.parametrize("prefix_zero", [False, True])
@pytest.mark.parametrize("shared,N,G,D", [(4, 5, 4, 1), (105, 11, 64, 4), (153, 9, 128, 3), (65, 3, 2, 1)])
def test_a_prefix_and_own_parts_of_unlike_sizes(shared, N, G, D, prefix_zero, up):
    c = build([shared * 16 + 40 + 33 * i for i in range(N)], shared=shared, Hkv=1, D=D, G=G, B=16, seed=9)
    check(zeros_beside(c, up, lambda b: (b < shared) == prefix_zero), 0.125)


@pytest.mark.parametrize("up", [-64, -50, 60, 118])
@pytest.mark.parametrize("Dh,Hkv,G,D", [(64, 4, 4, 1), (64, 2, 8, 4), (128, 1, 7, 1)])
def test_all_values_near_the_ends_of_the_range(Dh, Hkv, G, D, up):
    c = build([300, 45, 1024], D=D, G=G, Hkv=Hkv, Dh=Dh, B=8, seed=10)
    c["vs"][~np.isnan(c["vs"])] = np.float32(2.0 ** up)
    check(c, Dh ** -0.5)


def test_zeros_and_large_values_as_append_writes_them():
    x = torch.randn((96, 2, 64), generator=torch.Generator().manual_seed(11))
    v = x * 2.0 ** 100
    v[:48] = 0
    k, kv, ks, vs = sc.page_cache_8bit(6, 16, 2, 64, block=8)
    table, lens, slots = i32([[5, 3, 1, 0, 2, 4]]), i32([96]), i32([0])
    sc.pages_append(x.cuda(), v.cuda(), k, kv, table, lens, slots, 96, k_scales=ks, v_scales=vs)
    q = (x[-1:].repeat(1, 4, 1) * 0.5).bfloat16()
    c = dict(q=q, k=codes_from(k), v=codes_from(kv), ks=ks.cpu().numpy(), vs=vs.cpu().numpy(),
             table=table.cpu().numpy(), lens=np.array([96]), slots=np.array([0]), D=1, shared=0)
    assert c["vs"].min() == 2.0 ** -64 and c["vs"].max() > 2.0 ** 90
    check(c, 0.125)
