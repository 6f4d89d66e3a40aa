"""Rotary positions and their gradient on the GPU against the definition in float64, with exact angles.

The bound: a sine or cosine is off by at most 2 2^-24 of 1 (sincospif, 1 last place, of an angle whose
fraction of a turn is rounded once), a value is a sum of two products of fp32 numbers: |err| <= 6 2^-24
amplitude (|a| + |b|), and in bf16 half a step of the value, 2^-8 |value|, once more.
"""
import numpy as np
import pytest
import torch

import lfm2_gated_short_gb300 as sc
from cache8_util import i32
from oracle import cache8

pytestmark = pytest.mark.gpu


def bound(x, freqs, layout, amplitude, ref, dtype):
    R = 2 * len(freqs)
    mag = np.zeros(x.shape)
    a, b = (x[..., :R // 2], x[..., R // 2:R]) if layout == "half" else (x[..., 0:R:2], x[..., 1:R:2])
    s = amplitude * (np.abs(a) + np.abs(b))
    mag[..., :R] = np.concatenate([s, s], -1) if layout == "half" else np.repeat(s, 2, -1)
    return 6 * 2.0 ** -24 * mag + (2.0 ** -8 * np.abs(ref) if dtype is torch.bfloat16 else 0.0) * (mag > 0)


def check(T, Hq, Hkv, Dh, R, layout, dtype, positions, base=1e4, amplitude=1.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((T, Hq, Dh), generator=g).to(dtype)
    k = torch.randn((T, Hkv, Dh), generator=g).to(dtype)
    freqs, _ = sc.rope_frequencies(R, base=base)
    f = freqs.cpu().numpy()
    for call, inverse in ((sc.rope, False), (sc.rope_backward, True)):
        got = call(q.cuda(), k.cuda(), freqs, positions=i32(positions), layout=layout, amplitude=amplitude)
        assert sc.get_error() == 0
        for y, x in zip(got, (q, k)):
            x = x.double().numpy()
            ref = cache8.turned(x, positions, f, layout, amplitude, inverse)
            err = np.abs(y.double().cpu().numpy() - ref)
            assert (err <= bound(x, f, layout, amplitude, ref, dtype)).all(), err.max()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("Dh,R", [(64, 64), (64, 32), (64, 2), (128, 64), (80, 20), (80, 80), (96, 24),
                                  (256, 256), (512, 512), (7, 6), (66, 34)])
def test_heads_and_parts(dtype, layout, Dh, R):
    r = np.random.default_rng(R)
    check(9, 3, 2, Dh, R, layout, dtype, r.integers(0, 5000, 9), seed=R)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_positions_far_and_below_zero(dtype, layout):
    p = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 16777217, 1000003, -77777777]
    check(len(p), 2, 1, 64, 64, layout, dtype, p, amplitude=1.25)


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (1, 32, 8), (7, 5, 1), (130, 14, 2), (5000, 2, 1)])
def test_rows_and_heads(T, Hq, Hkv):
    check(T, Hq, Hkv, 64, 64, "half", torch.bfloat16, np.arange(T) + 11, base=1e6)


def test_frequencies_of_any_size():
    """Above a turn a position, tiny, zero and below zero."""
    f = np.array([7.5, 100.25, 1e-12, 0.0, -0.3, 2.0 ** 40 + 0.5, 1e-300, 2.0 ** 60])
    p = [0, 3, -9, 2 ** 31 - 1]
    x = np.random.default_rng(0).standard_normal((4, 1, 16)).astype(np.float32)
    got, _ = sc.rope(torch.from_numpy(x).cuda(), None, torch.from_numpy(f).cuda(), positions=i32(p))
    # A frequency's own 61 bits times the largest position leave 2^-28 turns of the large ones.
    few = [0, 1, 2, 3, 4, 6]
    ref = cache8.turned(x.astype(np.float64), p, f, "half")
    err = np.abs(got.double().cpu().numpy() - ref)
    lim = bound(x.astype(np.float64), f, "half", 1.0, ref, torch.float32)
    for i in few:
        turns = abs(f[i]) / (2 * np.pi)
        angle = 2 * np.pi * np.abs(p) * (2.0 ** -64 + (turns * 2.0 ** -61 if turns < 1 else turns * 2.0 ** -61))
        for j in (i, i + 8):
            extra = angle[:, None] * (np.abs(x[..., i]) + np.abs(x[..., i + 8]))
            assert (err[..., j] <= lim[..., j] + extra).all(), (i, err[..., j])
    assert np.isfinite(got.cpu().numpy()).all()


def test_large_frequencies_at_near_positions():
    """Thousands of turns and more a position: a frequency is held within 2^-61 of itself."""
    f = np.array([2.0 ** 20 + 0.3, 2.0 ** 30 + 0.25, 2.0 ** 40 + 0.5, 2.0 ** 52 + 1.0])
    p = [0, 1, -1, 2, 17, -1000]
    x = np.random.default_rng(1).standard_normal((6, 2, 8)).astype(np.float32)
    got, _ = sc.rope(torch.from_numpy(x).cuda(), None, torch.from_numpy(f).cuda(), positions=i32(p))
    ref = cache8.turned(x.astype(np.float64), p, f, "half")
    err = np.abs(got.double().cpu().numpy() - ref)
    lim = bound(x.astype(np.float64), f, "half", 1.0, ref, torch.float32)
    for i in range(4):
        angle = np.abs(p) * f[i] * 2.0 ** -61 + 2 * np.pi * np.abs(p) * 2.0 ** -64
        extra = angle[:, None] * (np.abs(x[..., i]) + np.abs(x[..., i + 4]))
        for j in (i, i + 4):
            assert (err[..., j] <= lim[..., j] + extra).all(), (i, err[..., j], extra)


def test_positions_of_cache_slots():
    D, lens, slots = 3, np.array([5, 3, 900, 70000]), [3, 0, 2]
    q = torch.randn((9, 4, 64)).cuda()
    k = torch.randn((9, 2, 64)).cuda()
    freqs, _ = sc.rope_frequencies(64)
    p = [lens[s] - D + j for s in slots for j in range(D)]
    a = sc.rope(q, k, freqs, lens=i32(lens), slot_ids=i32(slots), D=D)
    b = sc.rope(q, k, freqs, positions=i32(p))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and sc.get_error() == 0


def test_bad_slots_and_lengths_leave_rows_alone():
    q = torch.randn((8, 4, 64)).cuda()
    freqs, _ = sc.rope_frequencies(32)
    out = torch.full_like(q, 7.0)
    lens, slots = i32([50, 1, -4, 60]), i32([0, 1, 2, 9])
    sc.rope(q, None, freqs, lens=lens, slot_ids=slots, D=2, q_out=out)
    assert sc.get_error() == sc.DEV_BAD_SLOT | sc.DEV_BAD_LENGTH
    want, _ = sc.rope(q, None, freqs, positions=i32([48, 49, 0, 0, 0, 0, 0, 0]))
    assert torch.equal(out[:2], want[:2])
    assert (out[2] == 7.0).all() and torch.equal(out[3], want[3])  # a length of 1: its second row
    assert (out[4:] == 7.0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("R", [64, 32, 12])
def test_in_place_on_one_projection(dtype, layout, R):
    """q and k between each other's rows, turned in place; v and what R leaves out stay."""
    qkv = torch.randn((33, 8, 64), device="cuda").to(dtype)
    freqs, _ = sc.rope_frequencies(R)
    p = i32(np.arange(33) * 5)
    q, k, v = qkv.split((4, 2, 2), 1)
    want = sc.rope(q.contiguous(), k.contiguous(), freqs, positions=p, layout=layout)
    kept = qkv.clone()
    sc.rope(q, k, freqs, positions=p, layout=layout, q_out=q, k_out=k)
    assert sc.get_error() == 0
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(v, kept[:, 6:]) and torch.equal(qkv[..., R:], kept[..., R:])


def test_unaligned_rows():
    wide = torch.randn((5, 4 * 64 + 3), device="cuda")
    q = wide[:, 1:257].unflatten(1, (4, 64))
    freqs, _ = sc.rope_frequencies(64)
    p = i32([3, 9, 2, 0, 1])
    got, _ = sc.rope(q, None, freqs, positions=p)
    want, _ = sc.rope(q.contiguous(), None, freqs, positions=p)
    assert torch.allclose(got, want, rtol=0, atol=1e-6) and sc.get_error() == 0


def test_one_of_the_two():
    q, k = torch.randn((6, 4, 64)).cuda(), torch.randn((6, 2, 64)).cuda()
    freqs, _ = sc.rope_frequencies(64)
    p = i32(range(6))
    both = sc.rope(q, k, freqs, positions=p)
    only_q, none = sc.rope(q, None, freqs, positions=p)
    assert none is None and torch.equal(only_q, both[0])
    none, only_k = sc.rope(None, k, freqs, positions=p)
    assert none is None and torch.equal(only_k, both[1])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient_against_differences(layout):
    """The turn is linear: for fp32 inputs, <dy, f(x + e) - f(x)> = <f'(dy), e> up to rounding."""
    g = torch.Generator().manual_seed(3)
    x, e, dy = (torch.randn((20, 3, 32), generator=g).cuda() for _ in range(3))
    freqs, _ = sc.rope_frequencies(16)
    kw = dict(positions=i32(range(100, 120)), layout=layout, amplitude=1.2)
    a, b = sc.rope(x + e, None, freqs, **kw)[0], sc.rope(x, None, freqs, **kw)[0]
    dx = sc.rope_backward(dy, None, freqs, **kw)[0]
    e = ((x + e).double() - x.double())
    left, right = (dy.double() * (a.double() - b.double())).sum(), (dx.double() * e).sum()
    # 1920 terms of size about 1.2 with an error of 12 2^-24 each, added in 64 bits
    assert abs(float(left - right)) <= 1920 * 1.2 * 12 * 2.0 ** -24 * 4
