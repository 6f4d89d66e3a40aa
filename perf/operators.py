"""Measured cases of the speculative serving operators: the paged cache's fork, resize and compaction,
attention over it for a batch that shares a prefix, and the verification of drafted tokens.

A case's "op" says which: "pages_fork" (a fork of N branches and the room for their next tokens),
"pages_compact", "attention" (one step's keys and values appended, then the attention that reads them)
or "draft_accept". `own` False computes a case in plain torch operations, True with the library.
"""
import math

import numpy as np
import torch

own = False

# Row p of a cache layout: tokens of a page, kv heads, head width. H = 2048 as 32 heads of 64 is the
# width the repository's benchmark uses throughout.


def listed():
    return [
        # One stream without a shared prefix: the smallest decode step, where latency counts.
        dict(name="attn_one_stream", op="attention", N=1, D=1, Hkv=8, G=4, Dh=64, ps=16,
             shared=0, lo=1000, hi=1000),
        # Two long conversations decoded alone: the key axis has to be split to fill the GPU.
        dict(name="attn_long_pair", op="attention", N=2, D=1, Hkv=8, G=4, Dh=64, ps=32,
             shared=0, lo=30001, hi=40003),
        # An ordinary serving batch behind one system prompt, one token a sequence.
        dict(name="attn_batch_prompt", op="attention", N=64, D=1, Hkv=8, G=4, Dh=64, ps=16,
             shared=256, lo=64, hi=1500),
        # Odd counts, wide heads, few kv heads, three drafts a sequence.
        dict(name="attn_odd_wide", op="attention", N=37, D=3, Hkv=2, G=7, Dh=128, ps=32,
             shared=93, lo=3, hi=901),
        # Many samples of one long document, eight drafts a sequence: the largest.
        dict(name="attn_many_drafts", op="attention", N=128, D=8, Hkv=8, G=4, Dh=64, ps=64,
             shared=256, lo=100, hi=1200),
        # One sequence's drafts: latency.
        dict(name="accept_one", op="draft_accept", N=1, D=4, V=32000, dtype="f32", ragged=False,
             draft=True),
        # The serving verify step of the repository's benchmark (64 sequences, 8 drafts), 65536 tokens.
        dict(name="accept_batch", op="draft_accept", N=64, D=8, V=65536, dtype="f32", ragged=False,
             draft=True),
        # Large batch, odd vocabulary, bf16 probabilities, ragged draft counts.
        dict(name="accept_wide_bf16", op="draft_accept", N=256, D=5, V=130051, dtype="bf16",
             ragged=True, draft=True),
        # Two branches off a short prompt: latency.
        dict(name="fork_small", op="pages_fork", N=2, D=1, L=1, Hkv=8, Dh=64, ps=16, src_len=131,
             n_pages=256, busy=12),
        # 64 samples of a long prompt, 6 layers: 64 table rows of 1025 pages, 64 page copies a layer.
        dict(name="fork_batch", op="pages_fork", N=64, D=8, L=6, Hkv=8, Dh=64, ps=16,
             src_len=16391, n_pages=8192, busy=100),
        # A small pool squeezed.
        dict(name="compact_small", op="pages_compact", L=1, Hkv=8, Dh=64, ps=16, n_pages=301,
             n_slots=24, fill=0.5),
        # A large pool after many sequences have ended: 2 x 4 layers of 64 KB pages.
        dict(name="compact_large", op="pages_compact", L=4, Hkv=8, Dh=64, ps=64, n_pages=4096,
             n_slots=192, fill=0.55),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "draft_accept", "pages_fork", "pages_compact"])
    top = {"bytes": 0.0, "flops": 0.0}
    for c in listed():
        if c["op"] == op:
            w = work(c)
            top = {k: max(top[k], w[k]) for k in top}
    while True:
        if op == "attention":
            ps = rng.choice([16, 32, 64, 128])
            lo = _log_int(rng, 1, 4000)
            c = dict(op=op, N=_log_int(rng, 1, 200), D=rng.choice([1, 1, 2, 3, 5, 8]),
                     Hkv=rng.choice([1, 2, 4, 8]), G=rng.choice([1, 2, 4, 5, 7, 8]),
                     Dh=rng.choice([64, 128]), ps=ps,
                     shared=rng.choice([0, 1]) * (_log_int(rng, 64, 20000) // ps), lo=lo,
                     hi=lo + _log_int(rng, 1, 6000))
            c["lo"], c["hi"] = c["lo"] + c["D"], c["hi"] + c["D"]
        elif op == "draft_accept":
            c = dict(op=op, N=_log_int(rng, 1, 300), D=rng.choice([1, 2, 4, 5, 8]),
                     V=_log_int(rng, 1000, 160000), dtype=rng.choice(["f32", "bf16"]),
                     ragged=rng.choice([False, True]), draft=rng.choice([True, True, False]))
        elif op == "pages_fork":
            ps = rng.choice([16, 32, 64])
            src = _log_int(rng, 20, 16000)
            c = dict(op=op, N=_log_int(rng, 1, 64), D=rng.choice([1, 4, 8]),
                     L=rng.choice([1, 2, 6]), Hkv=rng.choice([2, 4, 8]), Dh=rng.choice([64, 128]),
                     ps=ps, src_len=src, n_pages=0, busy=_log_int(rng, 4, 100))
            c["n_pages"] = src // ps + 3 * c["N"] + 20 * c["busy"] + 16
        else:
            c = dict(op=op, L=rng.choice([1, 2, 4]), Hkv=rng.choice([2, 4, 8]),
                     Dh=rng.choice([64, 128]), ps=rng.choice([16, 32, 64]),
                     n_pages=_log_int(rng, 200, 6000), n_slots=_log_int(rng, 20, 200),
                     fill=rng.choice([0.3, 0.5, 0.7]))
        w = work(c)
        if all(w[k] <= top[k] for k in top):
            return c


def _own_lens(c, seed):
    """Own tokens of each sequence, the step's D among them, from a fixed generator."""
    g = np.random.RandomState(seed % 2**31)
    return g.randint(c["lo"], c["hi"] + 1, c["N"]).astype(np.int64)


def work(c):
    op = c["op"]
    if op == "attention":
        N, D, Hkv, G, Dh = c["N"], c["D"], c["Hkv"], c["G"], c["Dh"]
        P, mean = c["shared"] * c["ps"], (c["lo"] + c["hi"]) / 2
        token = Hkv * Dh * 2 * 2
        visible = P + mean - (D - 1) / 2
        return {"bytes": 2 * N * D * Hkv * G * Dh * 2 + (P + N * mean) * token + N * D * token * 2,
                "flops": 4.0 * Dh * Hkv * G * N * D * visible}
    if op == "draft_accept":
        es = 4 if c["dtype"] == "f32" else 2
        rows = 2 if c["draft"] else 1
        return {"bytes": float(c["N"] * (rows * c["V"] * es + (2 * c["D"] + 1) * 4 + 4 * c["D"])),
                "flops": float(c["N"] * rows * c["V"])}
    page = c["ps"] * c["Hkv"] * c["Dh"] * 2 * 2 * c["L"]  # K and V, all layers
    if op == "pages_fork":
        part = c["src_len"] % c["ps"]
        copied = c["N"] * page * part // c["ps"] * 2
        table = (c["N"] + 1) * (c["src_len"] // c["ps"] + 1) * 4
        return {"bytes": float(copied + table + 2 * c["n_pages"] * 4), "flops": 0.0}
    used = c["n_pages"] * c["fill"]
    movers = used * (1 - c["fill"])  # a used page's chance to lie past the used count
    return {"bytes": float(movers * page * 2 + 2 * (c["n_pages"] + used) * 4), "flops": 0.0}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def _normal(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _attention_state(c, seed):
    r, g = np.random.RandomState(seed % 2**31), _gen(seed)
    N, D, ps = c["N"], c["D"], c["ps"]
    own_len = _own_lens(c, seed)
    own_pages = -(-own_len // ps)
    most = -(-c["hi"] // ps)
    n_pages = c["shared"] + N * most + 5
    n_slots = N + 3
    max_pages = c["shared"] + most + 1
    ids = r.permutation(n_pages)
    table = np.full((n_slots, max_pages), -1, np.int64)
    lens = np.zeros(n_slots, np.int64)
    slots = r.permutation(n_slots)[:N]
    at = c["shared"]
    for i, s in enumerate(slots):
        table[s, :c["shared"]] = ids[:c["shared"]]
        table[s, c["shared"]:c["shared"] + own_pages[i]] = ids[at:at + own_pages[i]]
        lens[s] = c["shared"] * ps + own_len[i]
        at += own_pages[i]
    page = (n_pages, ps, c["Hkv"], c["Dh"])
    return dict(c, k_pages=_normal(page, g), v_pages=_normal(page, g),
                q=_normal((N * D, c["Hkv"] * c["G"], c["Dh"]), g) * 1.5,
                k=_normal((N * D, c["Hkv"], c["Dh"]), g), v=_normal((N * D, c["Hkv"], c["Dh"]), g),
                table=_dev(table), lens=_dev(lens), slots=_dev(slots))


def _accept_state(c, seed):
    g = _gen(seed)
    N, D, V = c["N"], c["D"], c["V"]
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    z = torch.randn((N, D + 1, V), generator=g, device="cuda") * 2.5
    target = torch.softmax(z, -1).to(dt)
    z = z[:, :D] + torch.randn((N, D, V), generator=g, device="cuda") * 0.7
    draft = torch.softmax(z, -1).to(dt) if c["draft"] else None
    noise = torch.rand((N, D, V), generator=g, device="cuda").clamp_(min=1e-7).log_().neg_().log_()
    tokens = (z - noise).argmax(-1).to(torch.int32)
    u = torch.rand((N, D + 1), generator=g, device="cuda")
    n = torch.randint(0, D + 1, (N,), generator=g, device="cuda", dtype=torch.int32)
    return dict(c, target=target, draft=draft, tokens=tokens, uniforms=u,
                n_drafts=n if c["ragged"] else None)


def _pool_state(c, seed, rows, n_slots, width):
    """Pools and a table whose slot s holds rows[s] tokens on pages spread over the pool."""
    r, g = np.random.RandomState(seed % 2**31), _gen(seed)
    ps, n_pages = c["ps"], c["n_pages"]
    need = [-(-t // ps) for t in rows]
    table = np.full((n_slots, width), -1, np.int64)
    lens = np.zeros(n_slots, np.int64)
    refs = np.zeros(n_pages, np.int64)
    ids, at = r.permutation(n_pages), 0
    for s, (t, n) in enumerate(zip(rows, need)):
        table[s, :n], lens[s] = ids[at:at + n], t
        refs[ids[at:at + n]] = 1
        at += n
    pool = (c["L"], n_pages, ps, c["Hkv"], c["Dh"])
    return dict(c, k_pages=_normal(pool, g), v_pages=_normal(pool, g), table=_dev(table),
                lens=_dev(lens), refs=_dev(refs))


def prepare(c, seed):
    if c["op"] == "attention":
        return _attention_state(c, seed)
    if c["op"] == "draft_accept":
        return _accept_state(c, seed)
    r = np.random.RandomState((seed + 1) % 2**31)
    if c["op"] == "pages_fork":  # slot 0 is forked to slots 1..N; the rest are other sequences
        N, ps = c["N"], c["ps"]
        rows = [c["src_len"]] + [0] * N + [int(x) for x in r.randint(1, 16 * ps, c["busy"])]
        width = max(16, -(-(c["src_len"] + c["D"]) // ps)) + 1
        s = _pool_state(c, seed, rows, 1 + N + c["busy"], width)
        s.update(src=_dev(np.zeros(N)), dst=_dev(np.arange(1, N + 1)),
                 new_lens=_dev(np.full(N, c["src_len"] + c["D"])))
        return s
    used = int(c["n_pages"] * c["fill"])
    cuts = np.sort(r.choice(np.arange(1, used), c["n_slots"] - 1, replace=False))
    pages = np.diff(np.concatenate([[0], cuts, [used]]))
    rows = [int(n) * c["ps"] - int(r.randint(0, c["ps"])) for n in pages]
    s = _pool_state(c, seed, rows, c["n_slots"], used - c["n_slots"] + 1)
    s.update(table0=s["table"].clone(), refs0=s["refs"].clone())
    return s


# ------------------------------------------------------------------ the operators in plain torch


def _plain_append(s):
    """Token j of sequence i goes to position lens - D + j of its slot."""
    D, ps = s["D"], s["ps"]
    slots = s["slots"].long()
    pos = s["lens"].long()[slots][:, None] - D + torch.arange(D, device="cuda")
    page = s["table"].long()[slots].gather(1, pos // ps)
    s["k_pages"][page.flatten(), (pos % ps).flatten()] = s["k"]
    s["v_pages"][page.flatten(), (pos % ps).flatten()] = s["v"]


def _plain_attention(s):
    """The prefix's scores once for all rows, the own keys' per sequence, one softmax over both."""
    N, D, Hkv, G, Dh, ps = (s[x] for x in ("N", "D", "Hkv", "G", "Dh", "ps"))
    slots = s["slots"].long()
    table, lens = s["table"].long()[slots], s["lens"].long()[slots]
    q = s["q"].float().view(N, D, Hkv, G, Dh) / math.sqrt(Dh)
    q = q.permute(2, 0, 1, 3, 4).reshape(Hkv, N, D * G, Dh)
    P = s["shared"] * ps
    front = table[0, :s["shared"]]
    kp = s["k_pages"][front].float().view(P, Hkv, Dh)
    vp = s["v_pages"][front].float().view(P, Hkv, Dh)
    mine = table[:, s["shared"]:].clamp(min=0)
    ko = s["k_pages"][mine].float().reshape(N, -1, Hkv, Dh)
    vo = s["v_pages"][mine].float().reshape(N, -1, Hkv, Dh)
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


def _weights(p):
    """Probabilities in whole units of 2^-40, so that their sums do not depend on the order."""
    return (p.float().clamp(0.0, 1.0) * 2.0**40).long()


def _plain_accept(s):
    """Accept tests in 64 bits (the product of two 32-bit numbers is exact there), sums in whole numbers."""
    N, D, V = s["N"], s["D"], s["V"]
    rows, js = torch.arange(N, device="cuda"), torch.arange(D, device="cuda")
    tokens, u = s["tokens"].long(), s["uniforms"]
    n = s["n_drafts"].long() if s["n_drafts"] is not None else torch.full_like(rows, D)
    px = s["target"][:, :D].gather(2, tokens[..., None])[..., 0].double()
    qx = 1.0
    if s["draft"] is not None:
        qx = s["draft"].gather(2, tokens[..., None])[..., 0].double()
    ok = (u[:, :D].double() * qx < px) & (js < n[:, None])
    a = ok.long().cumprod(1).sum(1)
    w = _weights(s["target"][rows, a])
    at = a.clamp(max=D - 1)
    if s["draft"] is not None:
        q = _weights(s["draft"][rows, at])
    else:
        q = torch.zeros_like(w).scatter_(1, tokens[rows, at][:, None], 2**40)
    rest = (w - q).clamp(min=0)
    rejected = (a < n) & (rest.sum(1) > 0)
    w = torch.where(rejected[:, None], rest, w)
    total, m = w.sum(1), (u[:, D] * 2.0**31).long()
    mark = (total >> 32) * m * 2 + (((total & 0xFFFFFFFF) * m) >> 31)
    pick = (w.cumsum(1) <= mark[:, None]).sum(1)
    j = torch.arange(D + 1, device="cuda")
    padded = torch.cat([tokens, torch.zeros_like(tokens[:, :1])], 1)
    out = torch.where(j < a[:, None], padded, torch.where(j == a[:, None], pick[:, None], -1))
    return a.to(torch.int32), out.to(torch.int32)


def _claim(refs, n):
    return (refs == 0).nonzero()[:, 0][:n]


def _plain_fork(s):
    ps, table, lens, refs = s["ps"], s["table"], s["lens"], s["refs"]
    src, dst = s["src"].long(), s["dst"].long()
    cols, n_pages = torch.arange(table.shape[1], device="cuda"), refs.shape[0]
    old = table[dst]
    refs -= torch.bincount(old[old >= 0].long(), minlength=n_pages).to(refs.dtype)
    full, part = lens[src] // ps, lens[src] % ps > 0
    rows = torch.where(cols < full[:, None], table[src], -1)
    refs += torch.bincount(rows[rows >= 0].long(), minlength=n_pages).to(refs.dtype)
    who = part.nonzero()[:, 0]
    new = _claim(refs, who.shape[0])
    last = table[src[who], full[who].long()].long()
    w, r = (torch.arange(ps, device="cuda") < (lens[src] % ps)[who][:, None]).nonzero(as_tuple=True)
    s["k_pages"][:, new[w], r] = s["k_pages"][:, last[w], r]
    s["v_pages"][:, new[w], r] = s["v_pages"][:, last[w], r]
    rows[who, full[who].long()] = new.to(rows.dtype)
    refs[new] = 1
    table[dst], lens[dst] = rows, lens[src]


def _plain_grow(s):
    """pages_resize of branches that only grow: the lowest free pages, in listed order."""
    ps, table, lens, refs = s["ps"], s["table"], s["lens"], s["refs"]
    dst, new_lens = s["dst"].long(), s["new_lens"]
    cols = torch.arange(table.shape[1], device="cuda")
    have, need = -(-lens[dst] // ps), -(-new_lens // ps)
    add = (cols >= have[:, None]) & (cols < need[:, None])
    rows = table[dst]
    new = _claim(refs, int(add.sum()))
    rows[add] = new.to(rows.dtype)
    refs[new] = 1
    table[dst], lens[dst] = rows, new_lens


def _plain_compact(s):
    table, refs = s["table"], s["refs"]
    used, ids = refs > 0, torch.arange(refs.shape[0], device="cuda")
    n = used.sum()
    movers, holes = (used & (ids >= n)).nonzero()[:, 0], (~used & (ids < n)).nonzero()[:, 0]
    s["k_pages"][:, holes], s["v_pages"][:, holes] = s["k_pages"][:, movers], s["v_pages"][:, movers]
    refs[holes] = refs[movers]
    refs[movers] = 0
    ids[movers] = holes
    table.copy_(torch.where(table >= 0, ids[table.clamp(min=0).long()].to(table.dtype), table))
    return n.to(torch.int32).view(1)


# ------------------------------------------------------------------ one pass


def run(s):
    if own:
        import lfm2_gated_short_gb300 as sc
    op = s["op"]
    if op == "attention":
        if own:
            sc.pages_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                            s["slots"], s["D"])
            out = sc.prefix_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                      s["slots"], s["D"], shared_pages=s["shared"])
        else:
            _plain_append(s)
            out = _plain_attention(s)
        return {"out": out, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if op == "draft_accept":
        if own:
            a, out = sc.draft_accept(s["target"], s["draft"], s["tokens"], s["uniforms"],
                                     n_drafts=s["n_drafts"])
        else:
            a, out = _plain_accept(s)
        return {"accepted": a, "tokens": out}
    n = None
    if op == "pages_fork":  # a second pass releases the branches of the first and forks again
        if own:
            sc.pages_fork(s["refs"], s["table"], s["lens"], s["src"], s["dst"], s["k_pages"],
                          s["v_pages"])
            sc.pages_resize(s["refs"], s["table"], s["lens"], s["dst"], s["new_lens"], s["k_pages"],
                            s["v_pages"])
        else:
            _plain_fork(s)
            _plain_grow(s)
    else:  # the fragmented pool's table and counts again, then the compaction
        s["table"].copy_(s["table0"])
        s["refs"].copy_(s["refs0"])
        if own:
            n = sc.pages_compact(s["refs"], s["table"], s["lens"], s["k_pages"], s["v_pages"])
        else:
            n = _plain_compact(s)
    return {"refs": s["refs"], "table": s["table"], "lens": s["lens"], "k_pages": s["k_pages"],
            "v_pages": s["v_pages"], "n_used": n}


# ------------------------------------------------------------------ the definitions in 64 bits


def _exact_attention(c, seed):
    s = _attention_state(c, seed)
    N, D, Hkv, G, Dh, ps = (s[x] for x in ("N", "D", "Hkv", "G", "Dh", "ps"))
    table, lens, slots = (s[x].cpu().numpy() for x in ("table", "lens", "slots"))
    out = torch.empty((N * D, Hkv * G, Dh), dtype=torch.float64, device="cuda")
    for i, slot in enumerate(slots):
        t = np.arange(lens[slot])
        page = torch.from_numpy(table[slot][t // ps]).long().cuda()
        row = torch.from_numpy(t % ps).cuda()
        keys, vals = s["k_pages"][page, row].double(), s["v_pages"][page, row].double()
        keys[-D:], vals[-D:] = s["k"][i * D:i * D + D].double(), s["v"][i * D:i * D + D].double()
        for j in range(D):
            n = int(lens[slot]) - D + j + 1
            q = s["q"][i * D + j].double().view(Hkv, G, Dh)
            z = torch.einsum("hgd,thd->hgt", q, keys[:n]) * Dh ** -0.5
            out[i * D + j] = torch.einsum("hgt,thd->hgd", torch.softmax(z, -1), vals[:n]).reshape(
                Hkv * G, Dh)
    return {"out": out, "k_pages": None, "v_pages": None}


def _exact_accept(c, seed):
    s = _accept_state(c, seed)
    N, D = c["N"], c["D"]
    tokens, u = s["tokens"].cpu().numpy(), s["uniforms"].double().cpu().numpy()
    count = s["n_drafts"].cpu().numpy() if s["n_drafts"] is not None else np.full(N, D)
    units = lambda row: np.floor(np.clip(row.double().cpu().numpy(), 0, 1) * 2.0**40).astype(object)  # noqa: E731
    accepted, out = np.zeros(N, np.int64), np.full((N, D + 1), -1, np.int64)
    for i in range(N):
        a = 0
        while a < count[i]:
            x = int(tokens[i, a])
            q = float(s["draft"][i, a, x].double()) if c["draft"] else 1.0
            if not u[i, a] * q < float(s["target"][i, a, x].double()):
                break
            out[i, a] = x
            a += 1
        p = units(s["target"][i, a])
        w = p
        if a < count[i]:
            q = units(s["draft"][i, a]) if c["draft"] else np.zeros(c["V"], object)
            if not c["draft"]:
                q[int(tokens[i, a])] = 1 << 40
            rest = np.maximum(p - q, 0)
            w = rest if rest.sum() else p
        mark = (int(w.sum()) * int(u[i, D] * 2.0**31)) >> 31
        accepted[i], out[i, a] = a, int(np.argmax(np.cumsum(w) > mark))
    return {"accepted": accepted, "tokens": out}


def exact(c, seed):
    if c["op"] == "attention":
        return _exact_attention(c, seed)
    if c["op"] == "draft_accept":
        return _exact_accept(c, seed)
    return None  # copies and whole numbers
