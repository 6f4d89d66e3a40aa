"""Plain definitions of the 8-bit cache and of rotary positions -- TEST INFRASTRUCTURE.

Numpy, in float64 and whole numbers, one loop a definition. An 8-bit cache is codes (uint8, e4m3)
``[n_pages, ps, Hkv, Dh]`` and scales (float32, powers of two) ``[n_pages, ps / B, Hkv]``. Only tests
may import this module, like the rest of ``oracle/``.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from oracle import serving

MIN_EXP, MAX_EXP = -64, 120
# 2 pi to 200 bits and more
TWO_PI = Fraction(
    62831853071795864769252867665590057683943387987502116419498891846156328125724, 10 ** 76)


def _decode_table():
    """The number of each of the 256 codes: sign, 4 bits of exponent (bias 7), 3 of mantissa."""
    out = np.zeros(256)
    for c in range(256):
        e, f = c >> 3 & 15, c & 7
        v = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        if c & 0x7F == 0x7F:
            v = np.nan
        out[c] = -v if c & 0x80 else v
    return out


DECODE = _decode_table()


def encode(y):
    """float64 numbers to codes: nearest, ties to even, up to 448 (infinities too), NaN 0x7F (its
    sign is not compared)."""
    y = np.asarray(y, np.float64)
    mag = np.minimum(np.abs(y), 448.0)
    ok = ~np.isnan(y)
    _, e = np.frexp(np.where(ok, mag, 0.0))
    last = np.exp2(np.maximum(e - 1, -6) - 3.0)
    steps = np.rint(np.where(ok, mag, 0.0) / last)  # a whole number of last places
    value = steps * last
    _, e = np.frexp(value)
    ex = np.maximum(e - 1, -6)
    m = np.rint(value / np.exp2(ex - 3.0)).astype(np.int64)  # 0 .. 15, 8 and up: normal
    code = np.where(m >= 8, ((ex + 7) << 3) | (m & 7), m)
    code = np.where(ok, code, 0x7F)
    return (code | np.where(np.signbit(y) & ok, 0x80, 0)).astype(np.uint8)


def held(scale):
    """What a scale's word stands for: its exponent, held to the range."""
    e = (np.asarray(scale, np.float32).view(np.uint32) >> 23 & 255).astype(np.int64) - 127
    return np.exp2(np.clip(e, MIN_EXP, MAX_EXP).astype(np.float64))


def scale_for(most):
    """The least power of two s with most <= 448 s, in the range."""
    e = MIN_EXP
    while Fraction(float(most)) > 448 * Fraction(2) ** e:
        e += 1
    return 2.0 ** min(e, MAX_EXP)


def values(codes, scales):
    """Pools as numbers."""
    B = codes.shape[1] // scales.shape[1]
    return DECODE[codes] * held(scales).repeat(B, axis=1)[..., None]


def append(codes, scales, x, table, lens, slots, D):
    """Rows ``x [N*D, Hkv, Dh]`` into one pool, in place; returns the error bits."""
    n_pages, ps, Hkv, _ = codes.shape
    B, err = ps // scales.shape[1], 0
    for i, s in enumerate(slots):
        if not 0 <= s < len(lens):
            err |= serving.BAD_SLOT
            continue
        n = int(lens[s])
        if not 0 <= n <= table.shape[1] * ps:
            err |= serving.BAD_LENGTH
            continue
        if n < D:
            err |= serving.BAD_LENGTH
        at = max(n - D, 0)
        while at < n:
            b0 = at // B * B
            to = min(n, b0 + B)
            page, r0 = table[s, b0 // ps], b0 % ps
            if not 0 <= page < n_pages:
                err |= serving.BAD_PAGE
                at = to
                continue
            for h in range(Hkv):
                new = np.asarray(x[i * D + at - (n - D):i * D + to - (n - D), h], np.float64)
                scale = scale_for(np.abs(new[np.isfinite(new)]).max(initial=0.0))
                if at > b0:
                    was = held(scales[page, r0 // B, h])
                    scale = max(scale, was)
                    old = codes[page, r0:r0 + at - b0, h]
                    if scale > was:
                        old[...] = encode(DECODE[old] * (was / scale))
                codes[page, r0 + at - b0:r0 + to - b0, h] = encode(new / scale)
                scales[page, r0 // B, h] = scale
            at = to
    return err


class Cache(serving.Cache):
    """The cache model with codes and scales in the place of values: ``k``, ``v`` ``[L, n_pages, ps,
    Hkv * Dh]`` uint8, ``ks``, ``vs`` ``[L, n_pages, ps / B, Hkv]``."""

    def __init__(self, n_slots, max_pages, n_pages, page_size, L, Hkv, Dh, B, rng):
        super().__init__(n_slots, max_pages, n_pages, page_size, L, Hkv * Dh)
        self.k, self.v = (rng.integers(0, 256, self.k.shape).astype(np.uint8) for _ in range(2))
        shape = (L, n_pages, page_size // B, Hkv)
        self.ks, self.vs = (np.exp2(rng.integers(-9, 3, shape)).astype(np.float32) for _ in range(2))

    def _copy(self, src, dst, rows):
        super()._copy(src, dst, rows)
        self.ks[:, dst], self.vs[:, dst] = self.ks[:, src], self.vs[:, src]


def turned(x, positions, freqs, layout, amplitude=1.0, inverse=False):
    """``x [T, H, Dh]`` with the first 2 len(freqs) values of each head turned, float64; angles
    reduced exactly."""
    x = np.array(x, np.float64)
    half = len(freqs)
    frac = np.array([[float(Fraction(int(p)) * Fraction(float(f)) / TWO_PI % 1) for f in freqs]
                     for p in positions]).reshape(len(positions), half)
    t = 2 * np.pi * frac * (-1.0 if inverse else 1.0)
    z = amplitude * np.exp(1j * t)[:, None]
    first = x[..., :2 * half]
    a, b = (first[..., :half], first[..., half:]) if layout == "half" else (first[..., 0::2],
                                                                           first[..., 1::2])
    w = (a + 1j * b) * z
    out = x.copy()
    if layout == "half":
        out[..., :half], out[..., half:2 * half] = w.real, w.imag
    else:
        out[..., 0:2 * half:2], out[..., 1:2 * half:2] = w.real, w.imag
    return out
