"""Caches in 8 bits for the tests: numpy codes and scales, and their tensors."""
import numpy as np
import torch

import lfm2_gated_short_gb300 as sc


def i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


def codes_to(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().view(torch.float8_e4m3fn)


def codes_from(t):
    return t.view(torch.uint8).cpu().numpy()


def same_codes(got, want):
    """Bit for bit, but for a NaN's sign."""
    nan = (want & 0x7F) == 0x7F
    return np.array_equal(got[~nan], want[~nan]) and ((got[nan] & 0x7F) == 0x7F).all()


def build(lens, shared=0, ps=16, B=16, Hkv=2, Dh=64, G=2, D=1, seed=0, spare=1, spread=1.0):
    """A cache whose listed sequences (random slots) share `shared` pages; whatever is past a
    sequence's end, and every unused page, holds NaN codes, and scales without a token NaN."""
    r = np.random.default_rng(seed)
    N = len(lens)
    own = [max(0, -(-int(n) // ps) - shared) for n in lens]
    n_pages, n_slots = shared + sum(own) + 3, N + 2
    max_pages = shared + max(own + [0]) + spare
    ids = r.permutation(n_pages)
    table = np.full((n_slots, max_pages), -1)
    slots, full = r.permutation(n_slots)[:N], np.zeros(n_slots, np.int64)
    pools = []
    for _ in range(2):
        codes = np.full((n_pages, ps, Hkv, Dh), 0x7F, np.uint8)
        scales = np.full((n_pages, ps // B, Hkv), np.nan, np.float32)
        pools.append((codes, scales))

    def fill(page, rows):
        for codes, scales in pools:
            x = torch.from_numpy(np.clip(r.standard_normal((rows, Hkv, Dh)) * 110 * spread, -448, 448))
            codes[page, :rows] = x.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            blocks = -(-rows // B)
            scales[page, :blocks] = np.exp2(r.integers(-9, -5, (blocks, Hkv)))
    for p in ids[:shared]:
        fill(p, ps)
    at = shared
    for i, s in enumerate(slots):
        table[s, :shared], full[s] = ids[:shared], lens[i]
        for e in range(own[i]):
            table[s, shared + e] = ids[at]
            fill(ids[at], min(ps, int(lens[i]) - (shared + e) * ps))
            at += 1
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((N * D, Hkv * G, Dh), generator=g) * 1.5).bfloat16()
    return dict(q=q, k=pools[0][0], ks=pools[0][1], v=pools[1][0], vs=pools[1][1], table=table, lens=full,
                slots=slots, D=D, shared=shared)


def on_device(c):
    return dict(k=codes_to(c["k"]), v=codes_to(c["v"]), ks=torch.from_numpy(c["ks"]).cuda(),
                vs=torch.from_numpy(c["vs"]).cuda(), table=i32(c["table"]), lens=i32(c["lens"]),
                slots=i32(c["slots"]), q=c["q"].cuda())


def attend(c, **kw):
    d = on_device(c)
    return sc.prefix_attention(d["q"], d["k"], d["v"], d["table"], d["lens"], d["slots"], c["D"],
                               shared_pages=c["shared"], k_scales=d["ks"], v_scales=d["vs"], **kw)
