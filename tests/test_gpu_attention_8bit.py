"""Attention over the 8-bit paged cache on the GPU against the definition in float64.

The bound, with w the weights, A = sum w |v| and eps = 2^-8, bf16's unit roundoff: codes times scales
are exact, queries too where f16 holds them (or within 2^-25 of their row's largest); a weight enters
the second product rounded to f16 (2^-11) or, of a shared prefix, to bf16 (eps relative), with an fp32
score behind it whose error moves it by less than eps / 4 at these inputs (|score| < 64: 64 2^-24
log2 steps, and 128 products of relative 2^-24); the sum it is divided by keeps the unrounded
weights, and out is rounded once: |err| <= 1.5 eps A + 1.01 eps |out|, plus 2^-40 for results near
zero.
"""
import numpy as np
import pytest
import torch

import lfm2_gated_short_gb300 as sc
from cache8_util import attend, build, i32, on_device
from oracle import cache8, serving

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -8


def reference(c, scale):
    k, v = (np.nan_to_num(cache8.values(c[x], c[x + "s"])) for x in "kv")
    return serving.attention(c["q"].double().numpy(), k, v, c["table"], c["lens"], c["slots"], c["D"],
                             scale)


def check(c, scale=None, **kw):
    ref, mag = reference(c, scale or c["q"].shape[2] ** -0.5)
    got = attend(c, scale=scale, **kw)
    assert sc.get_error() == 0
    got = got.double().cpu().numpy()
    over = np.abs(got - ref) - (1.5 * EPS * mag + 1.01 * EPS * np.abs(ref) + 2.0 ** -40)
    assert np.isfinite(got).all() and (over <= 0).all(), (np.abs(got - ref).max(), over.max())


EDGES = [0, 1, 2, 7, 8, 9, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257]


@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("ps,B", [(8, 8), (16, 8), (16, 16), (32, 16), (64, 64), (128, 8), (128, 128),
                                  (256, 32), (256, 256)])
def test_lengths_pages_and_blocks(Dh, ps, B):
    check(build(EDGES, ps=ps, B=B, Dh=Dh, seed=ps + Dh + B))


@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("Hkv,G,D", [(1, 1, 1), (8, 4, 1), (2, 7, 1), (1, 5, 3), (3, 16, 1), (2, 4, 8),
                                     (1, 33, 1), (2, 3, 21), (1, 128, 1), (1, 128, 3), (5, 2, 9)])
def test_heads_and_drafts(Dh, Hkv, G, D):
    check(build([40, 3, 129, 64, 300], Hkv=Hkv, G=G, D=D, Dh=Dh, seed=G + D))


@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("shared,ps,B,lens", [
    (1, 16, 16, [17, 30, 16]), (4, 16, 8, [64, 65, 66, 200]), (9, 16, 16, [150, 144, 301]),
    (8, 16, 16, [129, 128, 140, 1000]), (5, 32, 16, [161, 260]), (3, 64, 8, [200, 192, 193]),
    (2, 128, 64, [257, 256, 400]), (33, 8, 8, [265, 270, 264]), (65, 16, 16, [1041, 1100]),
    (1, 256, 256, [300])])
@pytest.mark.parametrize("D,G", [(1, 4), (5, 3)])
def test_shared_prefix(Dh, shared, ps, B, lens, D, G):
    check(build(lens, shared=shared, ps=ps, B=B, D=D, G=G, Dh=Dh, seed=shared))


def test_rows_that_end_inside_the_shared_part():
    c = build([64, 64, 64, 70], shared=4, D=3, seed=4)
    for i, n in enumerate((64, 50, 2)):
        c["lens"][c["slots"][i]] = n
    check(c)


@pytest.mark.parametrize("shared", [0, 40])
def test_many_rows(shared):
    r = np.random.default_rng(11)
    check(build(r.integers(641, 900, 70), shared=shared, D=4, G=4, seed=11))


@pytest.mark.parametrize("Dh,ps", [(64, 16), (128, 32)])
@pytest.mark.parametrize("N,D,G", [(17, 8, 4), (3, 1, 5)])
def test_long_shared_prefix(Dh, ps, N, D, G):
    n = 4096 // ps
    check(build([4096 + D + 3 * i for i in range(N)], shared=n, ps=ps, D=D, G=G, Hkv=1, Dh=Dh, seed=5))


# A prefix that many rows share is unpacked once; the workspace then has room for it.

def unpacked(lens, shared, **kw):
    c = build(lens, shared=shared, **kw)
    ps, Hkv, Dh = c["k"].shape[1:]
    need = [sc.prefix_attention_8bit_workspace_bytes(c["q"].shape[1], Hkv, Dh, len(lens), c["D"], n, ps)
            for n in (0, shared)]
    assert need[1] - need[0] >= 4 * shared * ps * Hkv * Dh
    return c


@pytest.mark.parametrize("Dh,Hkv,G,D,N,shared,ps,B", [
    (64, 2, 64, 4, 10, 105, 16, 16), (64, 1, 128, 3, 9, 153, 16, 8), (128, 1, 5, 9, 23, 23, 256, 128),
    (64, 8, 4, 1, 47, 17, 64, 8), (128, 3, 7, 2, 60, 101, 8, 8), (64, 4, 8, 8, 35, 69, 32, 32),
    (128, 5, 1, 1, 90, 27, 32, 16)])
def test_unpacked_prefix(Dh, Hkv, G, D, N, shared, ps, B):
    """Own parts of D tokens, to several tiles; ends on and around page and tile borders."""
    r = np.random.default_rng(G)
    own = [D, D + 1, ps, ps + 1, 64 + D, 129, *r.integers(D, 300, N)][:N]
    check(unpacked([shared * ps + max(n, D) for n in own], shared, Dh=Dh, Hkv=Hkv, G=G, D=D, ps=ps, B=B,
                   seed=N))


def test_rows_that_end_inside_an_unpacked_prefix():
    c = unpacked([105 * 16 + 20] * 11, 105, G=64, D=4, seed=31)
    for i, n in enumerate((105 * 16 + 3, 105 * 16, 900, 3, 0)):  # the first that sees all is the sixth
        c["lens"][c["slots"][i]] = n
    check(c)


def test_an_unpacked_prefix_with_bad_data():
    c = unpacked([105 * 16 + 20] * 11, 105, G=64, D=4, seed=32)
    ref, mag = reference(c, 0.125)
    d = on_device(c)
    for bad_page in (-1, len(c["k"]), 2 ** 31 - 1):
        slots, lens, table = c["slots"].copy(), c["lens"].copy(), c["table"].copy()
        slots[0], lens[slots[1]] = -5, -1
        table[slots[3], 105] = bad_page
        out = torch.full(d["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
        args = dict(shared_pages=105, k_scales=d["ks"], v_scales=d["vs"], out=out)
        sc.prefix_attention(d["q"], d["k"], d["v"], i32(table), i32(lens), i32(slots), 4, **args)
        assert sc.get_error() == sc.DEV_BAD_SLOT | sc.DEV_BAD_LENGTH | sc.DEV_BAD_PAGE
        got = out.double().cpu().numpy().reshape(11, 4, 128, 64)
        skipped = [0, 1, 3]
        assert (got[skipped] == 7.0).all()
        err = np.abs(got.reshape(ref.shape) - ref)
        ok = err <= 1.5 * EPS * mag + 1.01 * EPS * np.abs(ref) + 2.0 ** -40
        assert np.delete(ok.reshape(got.shape), skipped, 0).all()
        table[slots[2], 50] = bad_page  # in the prefix as the first good sequence has it: no row
        out.fill_(7.0)
        sc.prefix_attention(d["q"], d["k"], d["v"], i32(table), i32(lens), i32(slots), 4, **args)
        assert sc.get_error() & sc.DEV_BAD_PAGE
        assert (out == 7.0).all()


def test_an_unpacked_prefix_on_streams_and_in_graphs():
    cases = [unpacked([105 * 16 + 20 + 31 * i for i in range(11)], 105, G=64, D=4, seed=33 + i)
             for i in range(2)]
    dev = [on_device(c) for c in cases]

    def run(d, out=None):
        return sc.prefix_attention(d["q"], d["k"], d["v"], d["table"], d["lens"], d["slots"], 4,
                                   shared_pages=105, k_scales=d["ks"], v_scales=d["vs"], out=out)
    want = [run(d).clone() for d in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in dev]
    outs = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(4):
        for d, s, o in zip(dev, streams, outs):
            with torch.cuda.stream(s):
                run(d, o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    graph, x = torch.cuda.CUDAGraph(), {n: t.clone() for n, t in dev[0].items()}
    with torch.cuda.graph(graph):
        got = run(x)
    for d, w in zip(dev[::-1], want[::-1]):
        for n in ("q", "table", "lens", "slots"):
            x[n].copy_(d[n])
        for n in ("k", "v"):
            x[n].view(torch.uint8).copy_(d[n].view(torch.uint8))
        x["ks"].copy_(d["ks"])
        x["vs"].copy_(d["vs"])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, w)
    assert sc.get_error() == 0


@pytest.mark.parametrize("Dh", [64, 128])
def test_long_sequences_are_split(Dh):
    check(build([9000, 4001], Hkv=1, G=4, Dh=Dh, ps=64, B=32, seed=6))


def test_more_sequences_than_threads():
    r = np.random.default_rng(12)
    check(build(r.integers(0, 40, 700), Hkv=1, G=1, ps=8, B=8, seed=12))


def test_large_and_small_scales_and_queries():
    """Blocks of values from 2^-60 to 2^40 beside each other, queries from 2^-30 to 2^30 times
    their keys' inverse, rows of zeros: each row by its own sizes."""
    c = build([100, 200, 64], Hkv=2, G=3, B=8, seed=13)
    r = np.random.default_rng(13)
    live = ~np.isnan(c["vs"])
    c["vs"][live] = np.exp2(r.integers(-60, 40, live.sum()))
    check(c)
    c = build([100, 200, 64], Hkv=2, G=3, B=8, seed=14)
    c["ks"][~np.isnan(c["ks"])] = 2.0 ** -30
    c["q"] = (c["q"].float() * 2.0 ** 22).bfloat16()
    c["q"][0] = 0
    check(c)


def test_values_of_zero_in_a_block_alone():
    c = build([40, 17], B=8, seed=15)
    c["v"][:] = 0
    c["vs"][:] = 2.0 ** -64
    check(c)


@pytest.mark.parametrize("Dh,G", [(64, 2), (64, 9), (128, 2)])
def test_nan_in_a_later_draft_stays_with_the_rows_that_see_it(Dh, G):
    D = 3
    c = build([50, 9, 130], D=D, G=G, Dh=Dh, seed=16)
    for s in c["slots"]:
        t = int(c["lens"][s]) - 1  # the last draft: its own row alone sees it
        page, row = c["table"][s, t // 16], t % 16
        c["v"][page, row, :, 5] = 0xFF
        c["k"][page, row, :, 3] = 0x7F
    got = attend(c).double().cpu().numpy().reshape(3, D, -1, Dh)
    clean = dict(c, v=np.where(c["v"] == 0xFF, 0, c["v"]))
    k, v = (np.nan_to_num(cache8.values(clean[x], clean[x + "s"])) for x in "kv")
    ref, mag = serving.attention(c["q"].double().numpy(), k, v, c["table"], c["lens"], c["slots"], D,
                                 Dh ** -0.5)
    ref, mag = ref.reshape(got.shape), mag.reshape(got.shape)
    err = np.abs(got - ref)[:, :-1]
    assert (err <= 1.5 * EPS * mag[:, :-1] + 1.01 * EPS * np.abs(ref[:, :-1]) + 2.0 ** -40).all()
    assert np.isnan(got[:, -1]).all()


def test_strided_queries_and_given_outputs():
    c = build([40, 3, 129], seed=17)
    ref, mag = reference(c, 64 ** -0.5)
    wide = torch.full((3, 6, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 1:5] = c["q"].cuda()
    d = on_device(c)
    out = torch.empty((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(sc.prefix_attention_8bit_workspace_bytes(4, 2, 64, 3, 1, 0, 16), dtype=torch.uint8,
                     device="cuda")
    got = sc.prefix_attention(wide[:, 1:5], d["k"], d["v"], d["table"], d["lens"], d["slots"], 1,
                              k_scales=d["ks"], v_scales=d["vs"], out=out, workspace=ws)
    assert got is out and sc.get_error() == 0
    assert (np.abs(out.double().cpu().numpy() - ref) <= 1.5 * EPS * mag + 1.01 * EPS * np.abs(ref)).all()


@pytest.mark.parametrize("shared", [0, 2])
def test_bad_slots_lengths_and_pages_leave_rows_alone(shared):
    c = build([70, 70, 70, 70], shared=shared, seed=18)
    ref, mag = reference(c, 64 ** -0.5)
    d = on_device(c)
    slots, lens, table = c["slots"].copy(), c["lens"].copy(), c["table"].copy()
    lens[slots[1]] = table.shape[1] * 16 + 1
    table[slots[2], 3] = len(c["k"])
    slots[0] = 99
    out = torch.full((4, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    sc.prefix_attention(d["q"], d["k"], d["v"], i32(table), i32(lens), i32(slots), 1, shared_pages=shared,
                        k_scales=d["ks"], v_scales=d["vs"], out=out)
    assert sc.get_error() == sc.DEV_BAD_SLOT | sc.DEV_BAD_LENGTH | sc.DEV_BAD_PAGE
    got = out.double().cpu().numpy()
    assert (got[:3] == 7.0).all()
    assert (np.abs(got[3] - ref[3]) <= 1.5 * EPS * mag[3] + 1.01 * EPS * np.abs(ref[3]) + 2.0 ** -40).all()


def test_same_bits_every_time():
    c = build([900, 33, 2000], Hkv=2, G=4, D=2, seed=19)
    a = attend(c)
    for _ in range(3):
        assert torch.equal(a, attend(c))


@pytest.mark.parametrize("Dh,G,D", [(64, 4, 1), (64, 8, 2), (64, 8, 4), (128, 5, 3)])
def test_queries_that_are_not_finite_stay_in_their_rows(Dh, G, D):
    c = build([300, 45, 1, 0], Hkv=4, G=G, D=D, Dh=Dh, seed=20)
    clean = attend(c)
    rows = [(0, 1), (D, 0), (D, 2)]
    for (t, h), x in zip(rows, (float("nan"), float("inf"), -float("inf"))):
        c["q"][t, h, 3] = x
    got = attend(c)
    assert sc.get_error() == 0
    for t, h in rows:
        assert torch.isnan(got[t, h]).all()
        got[t, h] = clean[t, h]
    assert torch.equal(got, clean)
