"""The plain definitions of the 8-bit cache and of rotary positions against torch's conversions,
closed forms and each other."""
import numpy as np
import pytest
import torch

import lfm2_gated_short_gb300 as sc
from oracle import cache8


def test_codes_are_torchs_e4m3():
    x = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(cache8.DECODE, x, equal_nan=True)


def test_encode_rounds_like_a_conversion():
    r = np.random.default_rng(0)
    y = np.concatenate([r.standard_normal(4000) * np.exp2(r.integers(-12, 9, 4000)),
                        cache8.DECODE[:127], (cache8.DECODE[:126] + cache8.DECODE[1:127]) / 2,
                        [0.0, -0.0, 448.0, 449.0, 1e30, np.inf, -np.inf]])
    y = np.clip(y.astype(np.float32), -448, 448)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(cache8.encode(y), want)
    assert np.array_equal(cache8.encode([np.inf, -np.inf, np.nan, 500.0]) & 0x7F, [0x7E, 0x7E, 0x7F, 0x7E])


@pytest.mark.parametrize("most,scale", [(448.0, 1.0), (448.0001, 2.0), (224.0, 0.5), (0.0, 2.0 ** -64),
                                        (3.3e38, 2.0 ** 120), (1e-30, 2.0 ** -64), (1.0, 2.0 ** -8)])
def test_scale_is_the_least_that_fits(most, scale):
    assert cache8.scale_for(np.float32(most)) == scale


def test_append_keeps_values_near():
    """Values are within half a step of e4m3 (2^-4 relative, or 2^-10 of the scale), twice where a
    later append moved them."""
    r = np.random.default_rng(1)
    ps, B, Hkv, Dh = 16, 8, 2, 16
    codes, scales = np.zeros((8, ps, Hkv, Dh), np.uint8), np.ones((8, ps // B, Hkv), np.float32)
    table, lens, x = np.arange(8).reshape(2, 4), np.zeros(2, np.int64), [[], []]
    for D in (1, 3, 9, 1, 1, 20, 2):
        lens += D
        new = r.standard_normal((2 * D, Hkv, Dh)) * np.exp2(r.integers(-3, 4, (2 * D, 1, 1)))
        assert cache8.append(codes, scales, new, table, lens, [0, 1], D) == 0
        for i in range(2):
            x[i] += list(new[i * D:i * D + D])
    got = cache8.values(codes, scales)
    for i in range(2):
        t = np.arange(lens[i])
        want, have = np.array(x[i]), got[table[i][t // ps], t % ps]
        step = cache8.held(scales)[table[i][t // ps], t % ps // B][..., None]
        assert (np.abs(want - have) <= 2 * (2.0 ** -4 * np.abs(want) + 2.0 ** -10 * step)).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_turning_is_a_rotation(layout):
    r = np.random.default_rng(2)
    x, f = r.standard_normal((5, 2, 12)), np.array([1.0, 0.3, 0.01])
    p = [0, 1, 7, -3, 2000000000]
    y = cache8.turned(x, p, f, layout, 1.5)
    assert np.array_equal(y[0, :, 6:], x[0, :, 6:]) and np.allclose(y[0, :, :6], 1.5 * x[0, :, :6])
    back = cache8.turned(y, p, f, layout, 1 / 1.5, inverse=True)
    assert np.allclose(back, x, atol=1e-12)
    # the same two turns as one: q(m) . k(n) depends on m - n
    q, k = cache8.turned(x, [9] * 5, f, layout), cache8.turned(x[::-1], [4] * 5, f, layout)
    q5 = cache8.turned(x, [5] * 5, f, layout)
    assert np.allclose((q * k).sum(-1), (q5 * x[::-1]).sum(-1), atol=1e-12)


def test_frequencies():
    f, a = sc.rope_frequencies(8, base=100.0, device="cpu")
    assert a == 1.0 and f.dtype == torch.float64
    assert np.allclose(f.numpy(), 100.0 ** (-np.arange(0, 8, 2) / 8), rtol=1e-14)
    lin, _ = sc.rope_frequencies(8, base=100.0, scaling="linear", factor=4.0, device="cpu")
    assert np.allclose(lin.numpy() * 4, f.numpy(), rtol=1e-14)
    raised, _ = sc.rope_frequencies(8, base=100.0, scaling="base", factor=4.0, device="cpu")
    assert raised[0] == f[0] and np.isclose(float(raised[-1]) * 4, float(f[-1]), rtol=1e-12)
    parts, a = sc.rope_frequencies(64, base=1e4, scaling="parts", factor=8.0, device="cpu")
    full, _ = sc.rope_frequencies(64, base=1e4, device="cpu")
    ratio = (full / parts).numpy()
    assert ratio[0] == 1.0 and np.isclose(ratio[-1], 8.0) and (np.diff(ratio) >= -1e-12).all()
    assert np.isclose(a, 0.1 * np.log(8.0) + 1)
    for kw in (dict(R=7), dict(R=0), dict(R=8, scaling="other"), dict(R=8, factor=0.0),
               dict(R=8, base=-1.0)):
        with pytest.raises(ValueError):
            sc.rope_frequencies(device="cpu", **kw)


def test_a_raised_base_slows_every_pair_but_the_first():
    for R in (4, 6, 64):
        f, _ = sc.rope_frequencies(R, base=1e4, device="cpu")
        raised, a = sc.rope_frequencies(R, base=1e4, scaling="base", factor=4.0, device="cpu")
        ratio = (f / raised).numpy()
        assert a == 1.0 and ratio[0] == 1.0 and np.isclose(ratio[-1], 4.0, rtol=1e-12)
        assert (np.diff(ratio) > 0).all()
    for factor in (1.0, 4.0):  # the first pair is the only one
        with pytest.raises(ValueError):
            sc.rope_frequencies(2, scaling="base", factor=factor, device="cpu")
    for scaling in (None, "linear", "parts"):
        assert sc.rope_frequencies(2, scaling=scaling, factor=4.0, device="cpu")[0].shape == (1,)
