"""Attention over the 8-bit cache where weights lie far apart, against float64.

A channel in which the keys of most weight hold zero is made by the others alone, however small their
weights are beside the row's largest: the bound is channel by channel. It is that of
test_gpu_attention_8bit.py without the absolute term: a weight is rounded to 11 bits at worst (f16, or
8 bits, bf16, over an unpacked prefix), behind scores of less than 128 whose fp32 error moves it by
128 2^-24 log2 steps and 128 products of 2^-24, below eps / 4; out is rounded once:
|err| <= 1.5 eps sum w |v| + 1.01 eps |out|, eps = 2^-8.
"""
import numpy as np
import pytest
import torch

import lfm2_gated_short_gb300 as sc
from cache8_util import attend, build
from oracle import cache8, serving

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -8
LN2 = float(np.log(2.0))


def code(x):
    return cache8.encode(np.asarray(x, np.float64))


def check(c, scale, got=None):
    k, v = (np.nan_to_num(cache8.values(c[x], c[x + "s"])) for x in "kv")
    ref, mag = serving.attention(c["q"].double().numpy(), k, v, c["table"], c["lens"], c["slots"], c["D"],
                                 scale)
    got = attend(c, scale=scale) if got is None else got
    assert sc.get_error() == 0
    got = got.double().cpu().numpy()
    over = np.abs(got - ref) - (1.5 * EPS * mag + 1.01 * EPS * np.abs(ref))
    assert np.isfinite(got).all() and (over <= 0).all(), (
        (np.abs(got - ref) / np.maximum(mag, 1e-300)).max(), (over > 0).mean())


def peaked(lens, gap, up, alike, D=1, **kw):
    """Of every 16 keys one scores `gap` powers of two above the rest for a row of full size (rows are
    full, half, and more often than not a quarter or less); its block of 8 holds zeros but in
    channel 5, at a scale `up` powers of two above the others', which are held so that the rest's
    part comes out near one. `alike`: all the rest score the same."""
    c = build(lens, B=8, D=D, **kw)
    r = np.random.default_rng(gap + up)
    N, Hq, Dh = c["q"].shape
    ps = c["k"].shape[1]
    c["q"].zero_()
    size = torch.from_numpy(r.choice([1.0, 0.5, 0.25, 0.0], (N, Hq)))
    size[0] = 1.0
    c["q"][..., 0] = size.bfloat16()
    if not alike:
        c["q"][..., 1:9] = torch.from_numpy(r.standard_normal((N, Hq, 8)) / 8).bfloat16()
    live_k, live_v = c["k"] != 0x7F, c["v"] != 0x7F
    big = np.zeros(ps, bool)
    first = r.integers(0, 8)  # of its block
    for b in range(0, ps, 16):
        big[b:b + 8] = True
    c["k"][..., 0] = 0
    c["k"][:, first::16, :, 0] = code(gap)
    c["ks"][:] = 1.0
    rest = np.clip(r.standard_normal(c["k"][..., 1:].shape), -4, 4)
    c["k"][..., 1:] = np.where(live_k[..., 1:], code(rest), 0)
    v = c["v"]
    v[:, big] = np.where(np.arange(Dh) == 5, code(448.0), 0)
    v[:, ~big, :, 5] = 0
    low = np.float32(2.0 ** (gap - 8))
    c["vs"][:] = low
    c["vs"][:, ::2] = low * np.float32(2.0 ** up)
    dead = ~live_v.any(-1)  # past the sequences' ends
    c["v"][dead], c["k"][dead] = 0x7F, 0x7F
    return c


SHAPES = [(64, 1, 1, 1), (64, 2, 3, 2), (64, 4, 4, 1), (64, 1, 4, 4), (64, 2, 8, 4), (64, 4, 4, 8),
          (128, 1, 7, 1), (128, 4, 2, 1), (128, 4, 4, 3), (128, 2, 8, 4)]
GAPS = [(16, 0), (20, 0), (22, 0), (24, 0), (26, 0), (28, 0), (18, 8), (10, 14), (10, 20), (30, 16),
        (56, 8), (40, 64), (96, 0), (96, 8)]


@pytest.mark.parametrize("gap,up", GAPS)
@pytest.mark.parametrize("Dh,Hkv,G,D", SHAPES)
def test_small_weights_beside_a_large_one(Dh, Hkv, G, D, gap, up):
    check(peaked([300, 45, 1024, 17], gap, up, alike=gap % 4 == 0, D=D, G=G, Hkv=Hkv, Dh=Dh, seed=gap), LN2)


@pytest.mark.parametrize("gap,up", [(24, 0), (10, 14), (30, 16)])
@pytest.mark.parametrize("Dh,G,D", [(64, 4, 1), (64, 4, 4), (64, 8, 4), (128, 3, 1), (128, 4, 8)])
def test_many_tiles_a_part(Dh, G, D, gap, up):
    """Enough tiles that a CTA walks many, of several sequences."""
    r = np.random.default_rng(gap)
    check(peaked(r.integers(D, 700, 60), gap, up, alike=True, D=D, G=G, Hkv=4, Dh=Dh, seed=3), LN2)


def test_one_large_key_before_a_long_rest():
    """A first key of no value 20 powers of two above 40000 equal ones: theirs is the whole output."""
    c = build([40000], Hkv=1, G=4, ps=64, B=64, seed=5)
    c["q"].zero_()
    c["q"][..., 0] = 1.0
    c["k"][:], c["ks"][:], c["vs"][:] = 0, 1.0, 1.0
    c["v"][:] = code(np.random.default_rng(5).standard_normal(c["v"].shape))
    page = c["table"][c["slots"][0], 0]
    c["k"][page, 0, :, 0], c["v"][page, 0] = code(20.0), 0
    check(c, LN2)


@pytest.mark.parametrize("gap,up", [(24, 0), (10, 14)])
@pytest.mark.parametrize("Dh,G", [(64, 2), (64, 9), (128, 2)])
def test_small_weights_beside_a_nan_that_some_rows_do_not_see(Dh, G, gap, up):
    D = 3
    c = peaked([50, 9, 130], gap, up, alike=False, D=D, G=G, Dh=Dh, seed=6)
    clean = dict(c, v=c["v"].copy())
    for s in c["slots"]:
        t = int(c["lens"][s]) - 1
        c["v"][c["table"][s, t // 16], t % 16, :, 7] = 0xFF
    got = attend(c, scale=LN2).reshape(3, D, -1, Dh)
    assert sc.get_error() == 0
    want = attend(clean, scale=LN2).reshape(got.shape)
    assert torch.isnan(got[:, -1, :, 7]).all()
    k, v = (np.nan_to_num(cache8.values(clean[x], clean[x + "s"])) for x in "kv")
    ref, mag = (x.reshape(got.shape) for x in serving.attention(
        clean["q"].double().numpy(), k, v, clean["table"], clean["lens"], clean["slots"], D, LN2))
    for out in (got, want):
        err = np.abs(out.double().cpu().numpy() - ref)[:, :-1]
        assert (err <= 1.5 * EPS * mag[:, :-1] + 1.01 * EPS * np.abs(ref[:, :-1])).all()


def test_a_row_is_the_same_whatever_its_neighbours_weights():
    """Small weights in one row of a tile change no bit of the others."""
    c = peaked([300, 45, 1024], 24, 0, alike=False, D=2, G=4, Hkv=2, seed=7)
    c["q"][:, 1::2, 0] = 0.0
    a = attend(c, scale=LN2)
    c["q"][:, ::2, 0] = 0.0
    b = attend(c, scale=LN2)
    assert torch.equal(a[:, 1::2], b[:, 1::2]) and not torch.equal(a[:, ::2], b[:, ::2])
