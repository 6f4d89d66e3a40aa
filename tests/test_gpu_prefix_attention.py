"""Attention over the paged cache on the GPU against the definition in float64.

The bound, with w the weights, A = sum w |v| and eps = 2^-8, bf16's unit roundoff (8 significant
bits): a weight enters the second product rounded to bf16 (eps relative) with an fp32 score behind it
whose error moves it by less than eps / 4 at these inputs (|score| < 64: 64 2^-24 log2 steps, and
128 products of relative 2^-24), the sum it is divided by keeps the unrounded weights, and out is
rounded once: |err| <= 1.5 eps A + 1.01 eps |out|, plus 2^-40 for results near zero.
"""
import numpy as np
import pytest
import torch

import lfm2_gated_short_gb300 as sc
from oracle import serving

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -8


def i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


def build(lens, shared=0, ps=16, Hkv=2, Dh=64, G=2, D=1, seed=0, spare=1, junk=float("nan"), spread=1.0):
    """A cache whose listed sequences (random slots) share `shared` pages; whatever is past a
    sequence's end, and every unused page, holds `junk`."""
    r = np.random.default_rng(seed)
    N = len(lens)
    own = [max(0, -(-int(n) // ps) - shared) for n in lens]
    n_pages, n_slots = shared + sum(own) + 3, N + 2
    max_pages = shared + max(own + [0]) + spare
    ids = r.permutation(n_pages)
    table = np.full((n_slots, max_pages), -1)
    slots, full = r.permutation(n_slots)[:N], np.zeros(n_slots, np.int64)
    k = torch.full((n_pages, ps, Hkv, Dh), junk, dtype=torch.bfloat16)
    v = torch.full((n_pages, ps, Hkv, Dh), junk, dtype=torch.bfloat16)
    g = torch.Generator().manual_seed(seed)

    def fill(page, rows):
        k[page, :rows] = (torch.randn((rows, Hkv, Dh), generator=g) * spread).bfloat16()
        v[page, :rows] = torch.randn((rows, Hkv, Dh), generator=g).bfloat16()
    for p in ids[:shared]:
        fill(p, ps)
    at = shared
    for i, s in enumerate(slots):
        table[s, :shared], full[s] = ids[:shared], lens[i]
        for e in range(own[i]):
            table[s, shared + e] = ids[at]
            fill(ids[at], min(ps, int(lens[i]) - (shared + e) * ps))
            at += 1
    q = (torch.randn((N * D, Hkv * G, Dh), generator=g) * 1.5).bfloat16()
    return dict(q=q, k=k, v=v, table=table, lens=full, slots=slots, D=D, shared=shared)


def reference(c, scale):
    f = lambda t: t.double().numpy()  # noqa: E731
    return serving.attention(f(c["q"]), f(c["k"]), f(c["v"]), c["table"], c["lens"], c["slots"],
                             c["D"], scale)


def call(c, **kw):
    return sc.prefix_attention(c["q"].cuda(), c["k"].cuda(), c["v"].cuda(), i32(c["table"]),
                               i32(c["lens"]), i32(c["slots"]), c["D"], shared_pages=c["shared"], **kw)


def check(c, scale=None, **kw):
    ref, mag = reference(c, scale or c["q"].shape[2] ** -0.5)
    got = call(c, scale=scale, **kw)
    assert sc.get_error() == 0
    got = got.double().cpu().numpy()
    over = np.abs(got - ref) - (1.5 * EPS * mag + 1.01 * EPS * np.abs(ref) + 2.0 ** -40)
    assert np.isfinite(got).all() and (over <= 0).all(), (np.abs(got - ref).max(), over.max())


# One token to several tiles, ends on and around page and tile borders, an empty sequence.
EDGES = [0, 1, 2, 7, 8, 9, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200]


@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("ps", [8, 16, 32, 64, 128, 256])
def test_lengths_and_page_sizes(Dh, ps):
    check(build(EDGES, ps=ps, Dh=Dh, seed=ps + Dh))


@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("Hkv,G,D", [(1, 1, 1), (8, 4, 1), (2, 7, 1), (1, 5, 3), (3, 16, 1), (2, 4, 8),
                                     (1, 33, 1), (2, 3, 21), (1, 128, 1), (1, 128, 3)])
def test_heads_and_drafts(Dh, Hkv, G, D):
    check(build([40, 3, 129, 64], Hkv=Hkv, G=G, D=D, Dh=Dh, seed=G + D))


@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("shared,ps,lens", [
    (1, 16, [17, 30, 16]), (4, 16, [64, 65, 66, 200]), (9, 16, [150, 144, 301]),
    (8, 16, [129, 128, 140, 1000]), (5, 32, [161, 260]), (3, 64, [200, 192, 193]),
    (2, 128, [257, 256, 400]), (33, 8, [265, 270, 264]), (65, 16, [1041, 1100]), (1, 256, [300])])
@pytest.mark.parametrize("D,G", [(1, 4), (5, 3)])
def test_shared_prefix(Dh, shared, ps, lens, D, G):
    check(build(lens, shared=shared, ps=ps, D=D, G=G, Dh=Dh, seed=shared))


def test_rows_that_end_inside_the_shared_part():
    """Sequences no longer than the shared part (or shorter than D): their rows see their own keys only."""
    c = build([64, 64, 64, 70], shared=4, ps=16, D=3, seed=4)
    for i, n in enumerate((64, 50, 2)):
        c["lens"][c["slots"][i]] = n
    check(c)


@pytest.mark.parametrize("shared", [0, 40])
def test_many_rows_share_a_prefix(shared):
    r = np.random.default_rng(11)
    check(build(r.integers(641, 900, 70), shared=shared, D=4, G=4, Hkv=2, seed=11))


@pytest.mark.parametrize("Dh,ps", [(64, 16), (128, 32)])
@pytest.mark.parametrize("N,D,G", [(17, 8, 4), (3, 1, 5), (70, 1, 2)])
def test_long_shared_prefix(Dh, ps, N, D, G):
    """Many key tiles a CTA: every ring and buffer comes round several times."""
    r = np.random.default_rng(N)
    check(build(r.integers(20001, 20300, N), shared=20000 // ps, ps=ps, D=D, G=G, Hkv=1, Dh=Dh,
                seed=N))
    check(build(r.integers(3000, 3300, N), shared=3000 // ps, ps=ps, D=D, G=G, Hkv=6, Dh=Dh, seed=N))


@pytest.mark.parametrize("Dh,G", [(64, 4), (128, 7)])
def test_one_long_sequence(Dh, G):
    check(build([20001], ps=64, Hkv=2, G=G, Dh=Dh, seed=12))


def test_more_sequences_than_threads():
    r = np.random.default_rng(13)
    check(build(r.integers(0, 40, 700), ps=8, Hkv=1, G=1, seed=13))


@pytest.mark.parametrize("shared", [0, 8])
def test_large_scores(shared):
    """Scores to +-300 before the softmax: the running maximum moves and weights underflow. The
    score's own rounding (300 x 2^-17 log2 units) stays inside the bound's eps / 4."""
    check(build([200, 333, 150], shared=shared, D=2, seed=14, spread=16.0), scale=0.25)


def test_equal_scores_keep_the_mean():
    c = build([513, 129], seed=15)
    c["q"].zero_()
    check(c)


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), 3e38])
@pytest.mark.parametrize("shared", [0, 2])
def test_nothing_past_the_end_is_looked_at(junk, shared):
    check(build([37, 41, 100, 33], shared=shared, junk=junk, D=2, seed=16))


def test_strided_queries_and_given_buffers():
    c = build([37, 80], D=2, G=3, seed=17)
    ref = call(c)
    wide = torch.full((4, 6 * 64 + 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + 6 * 64] = c["q"].view(4, -1).cuda()
    q = wide[:, 8:8 + 6 * 64].unflatten(1, (6, 64))
    out = torch.empty_like(ref)
    ws = torch.full((sc.prefix_attention_workspace_bytes(6, 2, 64, 2, 2),), 255, dtype=torch.uint8,
                    device="cuda")
    got = sc.prefix_attention(q, c["k"].cuda(), c["v"].cuda(), i32(c["table"]), i32(c["lens"]),
                              i32(c["slots"]), 2, out=out, workspace=ws)
    assert got is out and torch.equal(out, ref)
    assert sc.get_error() == 0


@pytest.mark.parametrize("shared", [0, 20])
def test_the_same_call_gives_the_same_bits(shared):
    r = np.random.default_rng(18)
    c = build(r.integers(330, 2000, 40), shared=shared, D=2, G=4, seed=18)
    first = call(c)
    for _ in range(5):
        assert torch.equal(call(c), first)


def test_bad_data_leaves_its_rows_alone():
    c = build([100, 90, 80, 70], D=2, seed=19)
    ref, _ = reference(c, 0.125)
    for what in ("slot", "long", "negative", "page", "low page"):
        table, lens, slots = (np.array(c[x]) for x in ("table", "lens", "slots"))
        s = slots[1]
        if what == "slot":
            slots[1] = len(lens)
        elif what == "long":
            lens[s] = 10 ** 6
        elif what == "negative":
            lens[s] = -1
        else:
            table[s, 2] = 10 ** 6 if what == "page" else -1
        out = torch.full((8, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        call(dict(c, table=table, lens=lens, slots=slots), out=out)
        code = sc.get_error()
        assert code == (sc.DEV_BAD_SLOT if what == "slot" else sc.DEV_BAD_PAGE if "page" in what
                        else sc.DEV_BAD_LENGTH), what
        got = out.double().cpu().numpy()
        assert (got[2:4] == 7.0).all(), what
        rest = [0, 1, 4, 5, 6, 7]
        assert np.abs(got[rest] - ref[rest]).max() < 0.02, what


def test_offsets_past_32_bits():
    """A 5 GB pool whose used pages lie past 2^32 bytes, more than 2^31 elements in."""
    ps, Hkv, Dh, n_pages = 64, 8, 128, 41000
    k = torch.zeros((n_pages, ps, Hkv, Dh), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    c = build([100, 300], ps=ps, Hkv=Hkv, G=2, Dh=Dh, seed=20)
    n = c["k"].shape[0]
    k[-n:], v[-n:] = c["k"].cuda(), c["v"].cuda()
    table = np.where(c["table"] >= 0, c["table"] + n_pages - n, -1)
    got = sc.prefix_attention(c["q"].cuda(), k, v, i32(table), i32(c["lens"]), i32(c["slots"]), 1)
    assert sc.get_error() == 0
    assert torch.equal(got, call(c))


def test_on_another_stream():
    c = build([500, 300], seed=21)
    ref = call(c)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    args = (c["q"].cuda(), c["k"].cuda(), c["v"].cuda(), i32(c["table"]), i32(c["lens"]),
            i32(c["slots"]))
    ws = torch.empty(sc.prefix_attention_workspace_bytes(4, 2, 64, 2, 1), dtype=torch.uint8,
                     device="cuda")
    out = torch.empty_like(ref)
    torch.cuda.synchronize()
    sc.prefix_attention(*args, 1, out=out, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)
