"""Measured cases of a decoder's rotary positions and of its key/value cache in 8 bits: the rotation of
queries and keys and its gradient, the cache's quantising write, its reading back, and attention over it.

A case's "op" says which: "rope" (with "grad" the gradient too), "append", "read" or "attention". `own`
False computes a case in plain torch operations, True with the library.

The 8-bit cache: a pool [n_pages, ps, Hkv, Dh] of e4m3 codes beside scales [n_pages, ps / B, Hkv], powers of
two in 32 bits, one for every block of B tokens of a page and kv head; code times scale is the value. A
block's scale is the least with which all that was written to it fits.
"""
import math

import numpy as np
import torch

own = False
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # One token of each of 64 sequences, at the lengths that the cache holds: latency. The model
        # width is the one that the repository's benchmark uses, 32 heads of 64 and 8 kv heads.
        dict(name="rope_step", op="rope", T=64, D=1, Hkv=8, G=4, Dh=64, R=64, layout="half", dtype="bf16",
             base=1e6, scaling="none", far=30000, grad=False),
        # A training batch of packed sequences, forward and backward: the largest.
        dict(name="rope_train", op="rope", T=16384, D=0, Hkv=8, G=4, Dh=64, R=64, layout="half",
             dtype="bf16", base=1e6, scaling="none", far=0, grad=True),
        # Part of wide heads in pairs of neighbours, 32 bits, positions past a million, interpolated.
        dict(name="rope_far_part", op="rope", T=5001, D=0, Hkv=2, G=7, Dh=128, R=64, layout="interleaved",
             dtype="f32", base=1e4, scaling="parts", far=1100000, grad=True),
        # A decode step's keys and values, one token a sequence, most of them inside a block that
        # holds tokens already: latency.
        dict(name="append_step", op="append", N=64, D=1, Hkv=8, Dh=64, ps=16, B=16, dtype="bf16",
             lo=1, hi=2000),
        # A long prompt's.
        dict(name="append_prompt", op="append", N=1, D=16391, Hkv=8, Dh=64, ps=64, B=32, dtype="bf16",
             lo=16391, hi=16391),
        # A short conversation read back in 32 bits.
        dict(name="read_short", op="read", N=1, Hkv=2, Dh=128, ps=16, B=8, lo=131, hi=131, starts=False,
             dtype="f32"),
        # Sixteen long ones, each from somewhere inside on.
        dict(name="read_long", op="read", N=16, Hkv=8, Dh=64, ps=32, B=16, lo=2001, hi=9000, starts=True,
             dtype="bf16"),
        # One stream, one token: the smallest decode step, where latency counts.
        dict(name="attn8_one_stream", op="attention", N=1, D=1, Hkv=8, G=4, Dh=64, ps=16, B=16, shared=0,
             lo=1000, hi=1000),
        # Two long conversations decoded alone: the key axis has to be split to fill the GPU.
        dict(name="attn8_long_pair", op="attention", N=2, D=1, Hkv=8, G=4, Dh=64, ps=32, B=32, shared=0,
             lo=30001, hi=40003),
        # An ordinary serving batch of unlike lengths, one token a sequence.
        dict(name="attn8_batch", op="attention", N=128, D=1, Hkv=8, G=4, Dh=64, ps=16, B=16, shared=0,
             lo=200, hi=6000),
        # Odd counts, wide heads, few kv heads, three drafts a sequence behind a common prompt.
        dict(name="attn8_odd_wide", op="attention", N=37, D=3, Hkv=2, G=7, Dh=128, ps=32, B=8, shared=93,
             lo=3, hi=901),
        # Many samples of one long document, eight drafts a sequence: the most operations.
        dict(name="attn8_many_drafts", op="attention", N=128, D=8, Hkv=8, G=4, Dh=64, ps=64, B=64,
             shared=256, lo=100, hi=1200),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rope(rng):
    Dh = rng.choice([64, 64, 80, 96, 128])
    R = rng.choice([Dh, Dh, Dh // 2, Dh // 4])
    step = rng.choice([False, True])
    c = dict(op="rope", T=_log_int(rng, 1, 512 if step else 16384), D=0, Hkv=rng.choice([1, 2, 4, 8]),
             G=rng.choice([1, 2, 4, 5, 7, 8]), Dh=Dh, R=R, layout=rng.choice(["half", "interleaved"]),
             dtype=rng.choice(["bf16", "f32"]), base=rng.choice([1e4, 5e5, 1e6]),
             scaling=rng.choice(["none", "linear", "parts"]),
             far=_log_int(rng, 1000, 2000000) if step else rng.choice([0, _log_int(rng, 1000, 2000000)]),
             grad=not step)
    if step:
        c["D"] = rng.choice([1, 2, 5])
        c["T"] *= c["D"]
    return c


def _draw_page(rng):
    ps = rng.choice([16, 32, 64, 128])
    return dict(Hkv=rng.choice([1, 2, 4, 8]), Dh=rng.choice([64, 128]), ps=ps,
                B=rng.choice([b for b in (8, 16, 32, 64, 128) if b <= ps]))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "attention", "attention"])
    top = {"bytes": 0.0, "flops": 0.0}
    for c in listed():
        if c["op"] == op:
            w = work(c)
            top = {k: max(top[k], w[k]) for k in top}
    while True:
        if op == "rope":
            c = _draw_rope(rng)
        elif op == "append":
            c = dict(op=op, N=_log_int(rng, 1, 256), D=rng.choice([1, 1, 3, 8, _log_int(rng, 10, 16000)]),
                     dtype=rng.choice(["bf16", "f32"]), **_draw_page(rng))
            c["lo"] = c["D"] + rng.choice([0, _log_int(rng, 1, 1000)])
            c["hi"] = c["lo"] + _log_int(rng, 1, 2000)
        elif op == "read":
            c = dict(op=op, N=_log_int(rng, 1, 64), starts=rng.choice([False, True]),
                     dtype=rng.choice(["bf16", "f32"]), **_draw_page(rng))
            c["lo"] = _log_int(rng, 1, 4000)
            c["hi"] = c["lo"] + _log_int(rng, 1, 6000)
        else:
            c = dict(op=op, N=_log_int(rng, 1, 200), D=rng.choice([1, 1, 2, 3, 5, 8]),
                     G=rng.choice([1, 2, 4, 5, 7, 8]), **_draw_page(rng))
            c["shared"] = rng.choice([0, 0, 1]) * (_log_int(rng, 64, 20000) // c["ps"])
            c["lo"] = c["D"] + _log_int(rng, 1, 4000)
            c["hi"] = c["lo"] + _log_int(rng, 1, 6000)
        w = work(c)
        if all(w[k] <= top[k] for k in top):
            return c


def work(c):
    op = c["op"]
    if op == "rope":
        es = 2 if c["dtype"] == "bf16" else 4
        values = c["T"] * c["Hkv"] * (c["G"] + 1) * c["Dh"] * (2 if c["grad"] else 1)
        turned = values * c["R"] // c["Dh"]
        return {"bytes": float(values * 2 * es + c["T"] * 4), "flops": 3.0 * turned}
    width = c["Hkv"] * c["Dh"]
    if op == "append":
        es = 2 if c["dtype"] == "bf16" else 4
        tokens = c["N"] * c["D"]
        blocks = c["N"] * (1 + (c["D"] - 1) // c["B"])
        return {"bytes": float(2 * tokens * width * (es + 1) + 2 * blocks * c["Hkv"] * 4),
                "flops": 2.0 * tokens * width * 2}
    mean = (c["lo"] + c["hi"]) / 2
    if op == "read":
        es = 2 if c["dtype"] == "bf16" else 4
        tokens = c["N"] * mean / (2 if c["starts"] else 1)
        return {"bytes": float(2 * tokens * (width * (es + 1) + 4 * c["Hkv"] / c["B"])),
                "flops": 2.0 * tokens * width}
    P = c["shared"] * c["ps"]
    rows = c["N"] * c["D"] * c["Hkv"] * c["G"]
    keys = P + c["N"] * mean
    return {"bytes": float(2 * rows * c["Dh"] * 2 + 2 * keys * (width + 4 * c["Hkv"] / c["B"])),
            "flops": 4.0 * c["Dh"] * rows * (P + mean - (c["D"] - 1) / 2)}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def _normal(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _frequencies(c):
    """Radians a position of each pair, in 64 bits, and the factor on sines and cosines. "linear": all
    positions eight times nearer; "parts": pairs that turn rarely within 8192 positions eight times
    slower, those that turn often as they were, a ramp between."""
    f = c["base"] ** (-np.arange(0, c["R"], 2, dtype=np.float64) / c["R"])
    if c["scaling"] == "linear":
        return f / 8.0, 1.0
    if c["scaling"] == "parts":
        turns = 8192 * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return f * (keep + (1 - keep) / 8.0), 0.1 * math.log(8.0) + 1.0
    return f, 1.0


def _rope_state(c, seed):
    r, g = np.random.RandomState(seed % 2**31), _gen(seed)
    T, D, Hkv, Hq, dt = c["T"], c["D"], c["Hkv"], c["Hkv"] * c["G"], _dtype(c)
    f, amplitude = _frequencies(c)
    s = dict(c, freqs=_dev(f, torch.float64), amplitude=amplitude)
    if D:  # a serving step: views of one projection, positions from the cache's lengths
        N = T // D
        slots = r.permutation(N + 5)[:N]
        lens = np.zeros(N + 5, np.int64)
        lens[slots] = D + r.randint(0, c["far"], N)
        s.update(slots=_dev(slots), lens=_dev(lens))
        s["q"], s["k"], _ = _normal((T, Hq + 2 * Hkv, c["Dh"]), g, dt).split((Hq, Hkv, Hkv), 1)
        return s
    cuts = np.sort(r.choice(T, min(T, 1 + T // 1500), replace=False))  # packed sequences
    cuts[0] = 0
    at = np.arange(T)
    s["positions"] = _dev(at - cuts[np.searchsorted(cuts, at, "right") - 1] + c["far"])
    s["q"], s["k"] = _normal((T, Hq, c["Dh"]), g, dt), _normal((T, Hkv, c["Dh"]), g, dt)
    if c["grad"]:
        s["dq"], s["dk"] = _normal((T, Hq, c["Dh"]), g, dt), _normal((T, Hkv, c["Dh"]), g, dt)
    return s


def _pool(c, n_pages, g):
    """Codes and scales of a pool whose values are about normal, each block's with a size of its own."""
    codes = (_normal((n_pages, c["ps"], c["Hkv"], c["Dh"]), g, torch.float32) * 110).clamp_(-448, 448)
    e = torch.randint(-9, -5, (n_pages, c["ps"] // c["B"], c["Hkv"]), generator=g, device="cuda")
    return codes.to(E4M3), torch.exp2(e.float())


def _cache_state(c, seed, own_len, shared=0):
    """Sequences of shared * ps + own_len[i] tokens on pages spread over two pools."""
    r, g = np.random.RandomState(seed % 2**31), _gen(seed)
    N, ps = len(own_len), c["ps"]
    need = -(-own_len // ps)
    # An append gives its whole pools back: as many pages for every seed.
    n_pages = shared + (N * -(-c["hi"] // ps) if c["op"] == "append" else int(need.sum())) + 5
    n_slots = N + 3
    ids = r.permutation(n_pages)
    table = np.full((n_slots, shared + int(need.max()) + 1), -1, np.int64)
    lens = np.zeros(n_slots, np.int64)
    slots = r.permutation(n_slots)[:N]
    at = shared
    for i, s in enumerate(slots):
        table[s, :shared] = ids[:shared]
        table[s, shared:shared + need[i]] = ids[at:at + need[i]]
        lens[s] = shared * ps + own_len[i]
        at += need[i]
    k_pages, k_scales = _pool(c, n_pages, g)
    v_pages, v_scales = _pool(c, n_pages, g)
    return dict(c, k_pages=k_pages, v_pages=v_pages, k_scales=k_scales, v_scales=v_scales,
                table=_dev(table), lens=_dev(lens), slots=_dev(slots)), g


def prepare(c, seed):
    if c["op"] == "rope":
        return _rope_state(c, seed)
    # What is read back is as long for every seed.
    r = np.random.RandomState(7 if c["op"] == "read" else (seed + 1) % 2**31)
    own_len = r.randint(c["lo"], c["hi"] + 1, c["N"]).astype(np.int64)
    s, g = _cache_state(c, seed, own_len, c.get("shared", 0))
    if c["op"] == "append":  # views of one projection; each token's size of its own
        rows = c["N"] * c["D"]
        x = _normal((rows, 4 * c["Hkv"], c["Dh"]), g, torch.float32)
        x *= torch.exp2(torch.rand((rows, 1, 1), generator=g, device="cuda") * 3 - 1.5)
        x = x.to(_dtype(c))
        s["k"], s["v"] = x[:, 2 * c["Hkv"]:3 * c["Hkv"]], x[:, 3 * c["Hkv"]:]
    elif c["op"] == "read":
        start = r.randint(0, own_len // 2 + 1) if c["starts"] else np.zeros(c["N"], np.int64)
        cu = np.concatenate([[0], np.cumsum(own_len - start)])
        s.update(start=_dev(start) if c["starts"] else None, cu=_dev(cu), T=int(cu[-1]))
    else:
        s["q"] = _normal((c["N"] * c["D"], c["Hkv"] * c["G"], c["Dh"]), g) * 1.5
    return s


# ------------------------------------------------------------------ the operators in plain torch


def _plain_turn(s, x, sign):
    """The first R values of each head turned by sign times position times frequency."""
    if s["D"]:
        last = s["lens"].long()[s["slots"].long()][:, None]
        pos = (last - s["D"] + torch.arange(s["D"], device="cuda")).flatten()
    else:
        pos = s["positions"]
    angle = pos.double()[:, None] * s["freqs"] * sign
    cos, sin = (f.float()[:, None] * s["amplitude"] for f in (angle.cos(), angle.sin()))
    R, out = s["R"], x.float()
    if s["layout"] == "half":
        a, b = out[..., :R // 2], out[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = out[..., 0:R:2], out[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, out[..., R:]], -1).to(x.dtype)


def _plain_append_one(s, x, pages, scales):
    """Each sequence's blocks from the one that its first new token lies in to its last, as one window."""
    N, D, ps, B, Hkv, Dh = (s[k] for k in ("N", "D", "ps", "B", "Hkv", "Dh"))
    slots, n_pages = s["slots"].long(), pages.shape[0]
    end = s["lens"].long()[slots][:, None]
    first = end - D
    blocks = (D + 2 * B - 2) // B
    pos = first // B * B + torch.arange(blocks * B, device="cuda")
    there = pos < end
    old, new = pos < first, (pos >= first) & there
    row = s["table"].long()[slots].gather(1, (pos // ps).clamp(max=s["table"].shape[1] - 1))
    at = row.clamp(min=0, max=n_pages - 1) * ps + pos % ps
    was = pages.view(n_pages * ps, Hkv, Dh)[at].float().view(N, blocks, B, Hkv, Dh)
    src = (torch.arange(N, device="cuda")[:, None] * D + pos - first).clamp(min=0, max=N * D - 1)
    came = torch.where(new[..., None, None], x[src].float(), 0.0).view(N, blocks, B, Hkv, Dh)
    size = torch.where(came.isfinite(), came.abs(), 0.0).amax((2, 4))
    part, power = torch.frexp(size / 448.0)  # size = 448 part 2^power, part in [1/2, 1)
    need = torch.where(part > 0.5, power, power - 1).clamp(min=-64)
    need = torch.where(size > 0, need, -64).float().exp2()
    block_at = at.view(N, blocks, B)[..., 0] // B
    scale_was = scales.view(-1, Hkv)[block_at]
    keeps = old.view(N, blocks, B)[..., 0][..., None]
    scale = torch.where(keeps, torch.maximum(scale_was, need), need)
    step = scale[:, :, None, :, None]
    kept = was * (scale_was[:, :, None, :, None] / step)
    code = torch.where(old.view(N, blocks, B, 1, 1), kept, (came / step).clamp(-448, 448)).to(E4M3)
    touched = new.view(N, blocks, B).any(2)
    pages.view(torch.uint8).view(n_pages * ps, Hkv, Dh)[at[there]] = (
        code.view(torch.uint8).view(N, blocks * B, Hkv, Dh)[there])
    scales.view(-1, Hkv)[block_at[touched]] = scale[touched]


def _plain_values(pages, scales, which):
    """Pages `which` as numbers."""
    x, y = pages[which].float(), scales[which]
    return x * y.repeat_interleave(x.shape[-3] // y.shape[-2], -2)[..., None]


def _plain_read(s):
    cu, slots = s["cu"].long(), s["slots"].long()
    t = torch.arange(s["T"], device="cuda")
    i = torch.searchsorted(cu, t, right=True) - 1
    pos = t - cu[i] + (s["start"].long()[i] if s["start"] is not None else 0)
    page, row = s["table"].long()[slots[i], pos // s["ps"]], pos % s["ps"]
    got = []
    for x, y in ((s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"])):
        got.append((x.view(torch.uint8)[page, row].view(E4M3).float()
                    * y[page, row // s["B"]][..., None]).to(_dtype(s)))
    return got


def _plain_attention(s):
    """The prefix's scores once for all rows, the own keys' per sequence, one softmax over both."""
    N, D, Hkv, G, Dh, ps = (s[x] for x in ("N", "D", "Hkv", "G", "Dh", "ps"))
    slots = s["slots"].long()
    table, lens = s["table"].long()[slots], s["lens"].long()[slots]
    q = s["q"].float().view(N, D, Hkv, G, Dh) / math.sqrt(Dh)
    q = q.permute(2, 0, 1, 3, 4).reshape(Hkv, N, D * G, Dh)
    P = s["shared"] * ps
    front, mine = table[0, :s["shared"]], table[:, s["shared"]:].clamp(min=0)
    kp, vp = (_plain_values(s[a], s[b], front).view(P, Hkv, Dh)
              for a, b in (("k_pages", "k_scales"), ("v_pages", "v_scales")))
    ko, vo = (_plain_values(s[a], s[b], mine).reshape(N, -1, Hkv, Dh)
              for a, b in (("k_pages", "k_scales"), ("v_pages", "v_scales")))
    sp = (q.reshape(Hkv, N * D * G, Dh) @ kp.permute(1, 2, 0)).view(Hkv, N, D * G, P)
    so = q @ ko.permute(2, 0, 3, 1)
    seen = lens[:, None] - D + 1 + torch.arange(D, device="cuda")  # keys of row (i, j)
    seen = seen.repeat_interleave(G, 1)[None, :, :, None]
    sp = sp.masked_fill(torch.arange(P, device="cuda") >= seen, -math.inf)
    so = so.masked_fill(P + torch.arange(so.shape[-1], device="cuda") >= seen, -math.inf)
    top = so.amax(-1, keepdim=True)
    top = torch.maximum(top, sp.amax(-1, keepdim=True)) if P else top
    ep, eo = (sp - top).exp_(), (so - top).exp_()
    total = ep.sum(-1, keepdim=True) + eo.sum(-1, keepdim=True)
    out = (ep.view(Hkv, N * D * G, P) @ vp.permute(1, 0, 2)).view(Hkv, N, D * G, Dh)
    out = (out + eo @ vo.permute(2, 0, 1, 3)) / total
    out = out.view(Hkv, N, D, G, Dh).permute(1, 2, 0, 3, 4)
    return out.reshape(N * D, Hkv * G, Dh).to(torch.bfloat16)


# ------------------------------------------------------------------ one pass


def _run_rope(s):
    if own:
        import lfm2_gated_short_gb300 as sc
        where = dict(layout=s["layout"], amplitude=s["amplitude"])
        if s["D"]:
            where.update(lens=s["lens"], slot_ids=s["slots"], D=s["D"])
        else:
            where.update(positions=s["positions"])
        q, k = sc.rope(s["q"], s["k"], s["freqs"], **where)
        if not s["grad"]:
            return {"q": q, "k": k}
        dq, dk = sc.rope_backward(s["dq"], s["dk"], s["freqs"], **where)
        return {"q": q, "k": k, "dq": dq, "dk": dk}
    got = {"q": _plain_turn(s, s["q"], 1.0), "k": _plain_turn(s, s["k"], 1.0)}
    if s["grad"]:  # a rotation's gradient is the rotation back
        got.update(dq=_plain_turn(s, s["dq"], -1.0), dk=_plain_turn(s, s["dk"], -1.0))
    return got


def run(s):
    if own:
        import lfm2_gated_short_gb300 as sc
    op = s["op"]
    if op == "rope":
        return _run_rope(s)
    if op == "append":  # codes come back as e4m3 numbers, beside the scales that they stand times
        if own:
            sc.pages_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["slots"],
                            s["D"], k_scales=s["k_scales"], v_scales=s["v_scales"])
        else:
            _plain_append_one(s, s["k"], s["k_pages"], s["k_scales"])
            _plain_append_one(s, s["v"], s["v_pages"], s["v_scales"])
        return {x: s[x] for x in ("k_pages", "v_pages", "k_scales", "v_scales")}
    if op == "read":
        if own:
            k, v = sc.pages_read(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"],
                                 s["lens"], s["slots"], s["cu"], s["T"], starts=s["start"],
                                 dtype=_dtype(s))
        else:
            k, v = _plain_read(s)
        return {"k": k, "v": v}
    if own:
        out = sc.prefix_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["slots"],
                                  s["D"], shared_pages=s["shared"], k_scales=s["k_scales"],
                                  v_scales=s["v_scales"])
    else:
        out = _plain_attention(s)
    return {"out": out}


# ------------------------------------------------------------------ the definitions in 64 bits


def _exact_rope(c, seed):
    """Pairs as complex numbers, turned by a unit number (times the amplitude)."""
    s = _rope_state(c, seed)
    if c["D"]:
        ends = s["lens"].cpu().numpy()[s["slots"].cpu().numpy()]
        pos = np.concatenate([np.arange(n - c["D"], n) for n in ends])
    else:
        pos = s["positions"].cpu().numpy()
    f, amplitude = _frequencies(c)
    turn = torch.polar(torch.full((len(pos), len(f)), amplitude, dtype=torch.float64),
                       torch.from_numpy(pos[:, None] * f)).cuda()[:, None]
    out = {}
    for name, by in (("q", turn), ("k", turn), ("dq", turn.conj()), ("dk", turn.conj())):
        if name not in s:
            continue
        x = s[name].double()
        half = c["layout"] == "half"
        pairs = x[..., :c["R"]].unflatten(-1, (2, -1) if half else (-1, 2))
        pairs = pairs.transpose(-1, -2) if half else pairs
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * by)
        x = x.clone()
        x[..., :c["R"]] = (z.transpose(-1, -2) if half else z).flatten(-2)
        out[name] = x
    return out


def _round_e4m3(y):
    """To the nearest number with 4 significant bits and a last place of 2^-9 at least, ties to even, up to 448."""
    _, e = np.frexp(np.abs(y))
    last = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.clip(np.round(y / last) * last, -448.0, 448.0)


def _exact_append(c, seed):
    s = prepare(c, seed)
    table, lens, slots = (s[x].cpu().numpy() for x in ("table", "lens", "slots"))
    got = {}
    for name in ("k", "v"):
        codes, scales = s[name + "_pages"].double().cpu().numpy(), s[name + "_scales"].double().cpu().numpy()
        x = s[name].double().cpu().numpy()
        for i, slot in enumerate(slots):
            n = int(lens[slot])
            at = n - c["D"]
            while at < n:  # block after block
                b0 = at // c["B"] * c["B"]
                to = min(n, b0 + c["B"])
                page, r0 = table[slot, b0 // c["ps"]], b0 % c["ps"]
                new = x[i * c["D"] + at - (n - c["D"]):i * c["D"] + to - (n - c["D"])]
                most = np.abs(new).max((0, 2))
                scale = np.exp2(np.maximum(np.ceil(np.log2(np.maximum(most, 1e-30) / 448.0)), -64))
                # log2 in 64 bits may be off beside a power of two: the definition itself decides
                scale = np.where(most > 448.0 * scale, scale * 2, scale)
                scale = np.where((most <= 224.0 * scale) & (scale > 2.0**-64), scale / 2, scale)
                was = scales[page, r0 // c["B"]].copy()
                if at > b0:
                    scale = np.maximum(scale, was)
                    codes[page, r0:r0 + at - b0] = _round_e4m3(
                        codes[page, r0:r0 + at - b0] * (was / scale)[:, None])
                codes[page, r0 + at - b0:r0 + to - b0] = _round_e4m3(new / scale[:, None])
                scales[page, r0 // c["B"]] = scale
                at = to
        got[name + "_pages"], got[name + "_scales"] = torch.from_numpy(codes), torch.from_numpy(scales)
    return got


def _exact_sequence(s, slot, pages, scales):
    """All tokens of a sequence as numbers in 64 bits."""
    t = np.arange(int(s["lens"][slot]))
    page = s["table"][slot].cpu().numpy()[t // s["ps"]]
    x = pages.double()[torch.from_numpy(page).cuda(), torch.from_numpy(t % s["ps"]).cuda()]
    y = scales.cpu().numpy()[page, t % s["ps"] // s["B"]].astype(np.float64)
    return x * torch.from_numpy(y).cuda()[..., None]


def _exact_read(c, seed):
    s, out = prepare(c, seed), {}
    cu = s["cu"].tolist()
    start = s["start"].tolist() if c["starts"] else [0] * c["N"]
    for name in ("k", "v"):
        rows = [_exact_sequence(s, slot, s[name + "_pages"], s[name + "_scales"])[a:a + cu[i + 1] - cu[i]]
                for i, (slot, a) in enumerate(zip(s["slots"].tolist(), start))]
        out[name] = torch.cat(rows)
    return out


def _exact_attention(c, seed):
    s = prepare(c, seed)
    N, D, Hkv, G, Dh = (s[x] for x in ("N", "D", "Hkv", "G", "Dh"))
    out = torch.empty((N * D, Hkv * G, Dh), dtype=torch.float64, device="cuda")
    k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
    for i, slot in enumerate(s["slots"].tolist()):
        keys = _exact_sequence(s, slot, k_pages, s["k_scales"])
        vals = _exact_sequence(s, slot, v_pages, s["v_scales"])
        for j in range(D):
            n = keys.shape[0] - D + j + 1
            q = s["q"][i * D + j].double().view(Hkv, G, Dh)
            z = torch.einsum("hgd,thd->hgt", q, keys[:n]) * Dh ** -0.5
            out[i * D + j] = torch.einsum("hgt,thd->hgd", torch.softmax(z, -1), vals[:n]).reshape(
                Hkv * G, Dh)
    return {"out": out}


def exact(c, seed):
    return dict(rope=_exact_rope, append=_exact_append, read=_exact_read,
                attention=_exact_attention)[c["op"]](c, seed)
