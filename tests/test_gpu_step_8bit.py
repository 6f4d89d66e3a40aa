"""Rotary positions and the 8-bit cache together, as a serving step uses them: rope at the cache's
lengths, a quantising append, attention over what was written, forks and rollbacks; on streams, in CUDA
graphs and from several host threads."""
import threading

import numpy as np
import pytest
import torch

import lfm2_gated_short_gb300 as sc
from cache8_util import codes_from, codes_to, i32, same_codes
from oracle import cache8, serving

pytestmark = pytest.mark.gpu

Hq, Hkv, Dh, EPS = 8, 2, 64, 2.0 ** -8


def new_cache(N, pages, n_pages, ps=16, B=8, layers=2):
    refs, table, lens = sc.page_cache(N, pages, n_pages)
    k, v, ks, vs = sc.page_cache_8bit(n_pages, ps, Hkv, Dh, block=B, layers=layers)
    return dict(refs=refs, table=table, lens=lens, k=k, v=v, ks=ks, vs=vs)


def scales(s, layer=None):
    pick = (lambda t: t) if layer is None else (lambda t: t[layer])
    return dict(k_scales=pick(s["ks"]), v_scales=pick(s["vs"]))


def resize(s, slots, lens):
    sc.pages_resize(s["refs"], s["table"], s["lens"], slots, lens, s["k"], s["v"], **scales(s))


def step(s, qkv, slots, D, freqs, amplitude, shared=0, stream=None):
    """All layers of one step on `qkv [layers, N*D, Hq + 2 Hkv, Dh]`, turned in place."""
    outs = []
    for l in range(s["k"].shape[0]):
        q, k, v = qkv[l].split((Hq, Hkv, Hkv), 1)
        sc.rope(q, k, freqs, lens=s["lens"], slot_ids=slots, D=D, amplitude=amplitude, q_out=q, k_out=k,
                stream=stream)
        sc.pages_append(k, v, s["k"][l], s["v"][l], s["table"], s["lens"], slots, D, stream=stream,
                        **scales(s, l))
        outs.append(sc.prefix_attention(q, s["k"][l], s["v"][l], s["table"], s["lens"], slots, D,
                                        shared_pages=shared, stream=stream, **scales(s, l)))
    return outs


def test_a_run_of_steps_against_the_definitions():
    """A prompt, a fork, steps with drafts and rollbacks, a compaction, in three layers of an odd number
    of pages (whose scales then start on no 16 bytes): every output, code and scale."""
    r = np.random.default_rng(0)
    ps, B, L, N, D = 16, 16, 3, 4, 3
    s = new_cache(N + 1, 12, 45, ps, B, L)
    assert s["ks"][1].data_ptr() % 16 != 0 or s["ks"][2].data_ptr() % 16 != 0
    m = cache8.Cache(N + 1, 12, 45, ps, L, Hkv, Dh, B, r)
    for t, a in ((s["k"], m.k), (s["v"], m.v)):
        t.copy_(codes_to(a).view(t.shape))
    for t, a in ((s["ks"], m.ks), (s["vs"], m.vs)):
        t.copy_(torch.from_numpy(a))
    freqs, amplitude = sc.rope_frequencies(32, scaling="parts", factor=8.0, original_length=64)
    f = freqs.cpu().numpy()

    def model_step(qkv, turned, slots, D):
        """The definitions on the GPU's own turned queries and keys (turning is tested by itself)."""
        pos = [m.lens[i] - D + j for i in slots for j in range(D)]
        refs = []
        for l in range(L):
            x, y = qkv[l].double().numpy(), turned[l].double().numpy()
            ref = cache8.turned(x[:, :Hq + Hkv], pos, f, "half", amplitude)
            a, b = np.abs(x[..., :16]), np.abs(x[..., 16:32])
            bound = 2.0 ** -8 * np.abs(ref)
            bound[..., :32] += 6 * 2.0 ** -24 * amplitude * np.concatenate([a + b, a + b], -1)[:, :Hq + Hkv]
            assert (np.abs(y[:, :Hq + Hkv] - ref) <= bound).all()
            assert np.array_equal(y[:, Hq + Hkv:], x[:, Hq + Hkv:])
            view = (45, ps, Hkv, Dh)
            for codes, sca, z in ((m.k, m.ks, y[:, Hq:Hq + Hkv]), (m.v, m.vs, y[:, Hq + Hkv:])):
                assert cache8.append(codes[l].reshape(view), sca[l], z, m.table, m.lens, slots, D) == 0
            k, v = (np.nan_to_num(cache8.values(c[l].reshape(view), z[l]))
                    for c, z in ((m.k, m.ks), (m.v, m.vs)))
            refs.append(serving.attention(y[:, :Hq], k, v, m.table, m.lens, slots, D, Dh ** -0.5))
        return refs

    def both(slots, D, shared=0):
        g = torch.Generator().manual_seed(int(m.lens.sum()))
        size = torch.exp2(torch.randint(-3, 4, (L, len(slots) * D, 1, 1), generator=g))
        qkv = (torch.randn((L, len(slots) * D, Hq + 2 * Hkv, Dh), generator=g) * size).bfloat16()
        qkv[:, :, :Hq] = torch.randn((L, len(slots) * D, Hq, Dh), generator=g).bfloat16()
        turned = qkv.cuda()
        outs = step(s, turned, i32(slots), D, freqs, amplitude, shared)
        refs = model_step(qkv, turned.cpu(), slots, D)
        assert sc.get_error() == 0
        for got, (ref, mag) in zip(outs, refs):
            # A score of at most 2^8 log2 steps has an error of 2^-16 of them: an eighth of eps / 4.
            over = np.abs(got.double().cpu().numpy() - ref) - (1.5 * EPS * mag + 1.01 * EPS * np.abs(ref))
            assert (over <= 2.0 ** -40).all(), over.max()
        check()

    def check():
        for name in ("refs", "table", "lens"):
            assert np.array_equal(s[name].cpu().numpy(), getattr(m, name)), name
        for t, a in ((s["k"], m.k), (s["v"], m.v)):
            assert same_codes(codes_from(t).reshape(a.shape), a)
        for t, a in ((s["ks"], m.ks), (s["vs"], m.vs)):
            assert np.array_equal(t.cpu().numpy(), a)

    def grow(slots, lens):
        resize(s, i32(slots), i32(lens))
        assert m.resize(slots, lens) == 0

    grow([0], [70])
    both([0], 70)  # the prompt
    slots = [1, 2, 3, 4]
    sc.pages_fork(s["refs"], s["table"], s["lens"], i32([0] * N), i32(slots), s["k"], s["v"], **scales(s))
    assert m.fork([0] * N, slots) == 0
    grow([0], [0])
    for _ in range(5):
        grow(slots, m.lens[slots] + D)
        both(slots, D, shared=4)
        grow(slots, m.lens[slots] - r.integers(0, D, N))
    used = sc.pages_compact(s["refs"], s["table"], s["lens"], s["k"], s["v"], **scales(s))
    assert int(used) == m.compact()
    check()
    grow(slots, m.lens[slots] + 1)
    both(slots, 1, shared=4)


def prepared(seed, N=6, D=2, base=200):
    """A cache with N sequences, and a step's projections."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = new_cache(N, 40, N * 40 + 3)
    slots = i32(np.random.default_rng(seed).permutation(N))
    lens = torch.randint(1, base, (N,), generator=g, device="cuda", dtype=torch.int32)
    resize(s, slots, lens)
    for t in (s["k"], s["v"]):
        t.view(torch.uint8).random_(0, 0x70, generator=g)
    for t in (s["ks"], s["vs"]):
        t.copy_(torch.exp2(torch.randint(-9, -5, t.shape, generator=g, device="cuda").float()))
    resize(s, slots, lens + D)
    qkv = torch.randn((2, N * D, Hq + 2 * Hkv, Dh), generator=g, device="cuda").bfloat16()
    return s, qkv, slots, D


def copy_of(s):
    return {n: t.view(torch.uint8).clone().view(t.dtype) if t.dtype == torch.float8_e4m3fn else t.clone()
            for n, t in s.items()}


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_on_streams_given_and_current():
    freqs, _ = sc.rope_frequencies(64)
    cases = [prepared(seed) for seed in range(4)]
    want = []
    for s, qkv, slots, D in cases:
        s = copy_of(s)
        want.append((step(s, qkv.clone(), slots, D, freqs, 1.0), s))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for rep in range(4):
        states = [copy_of(c[0]) for c in cases]
        inputs = [c[1].clone() for c in cases]
        torch.cuda.synchronize()
        got = []
        for (_, _, slots, D), s, qkv, st in zip(cases, states, inputs, streams):
            if rep % 2:
                got.append(step(s, qkv, slots, D, freqs, 1.0, stream=st))
            else:
                with torch.cuda.stream(st):
                    got.append(step(s, qkv, slots, D, freqs, 1.0))
        torch.cuda.synchronize()
        for outs, s, (ref, after) in zip(got, states, want):
            assert all(same(a, b) for a, b in zip(outs, ref))
            assert all(same(s[n], after[n]) for n in s)
    assert sc.get_error() == 0


def test_two_captured_steps_that_share_a_workspace():
    """Two graphs, replayed in turns on new inputs, with one workspace between them."""
    freqs, _ = sc.rope_frequencies(64)
    cases = [prepared(seed, N=5, D=3) for seed in (20, 21)]
    need = sc.prefix_attention_8bit_workspace_bytes(Hq, Hkv, Dh, 5, 3, 0, 16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def run(s, qkv, slots, D):
        q, k, v = qkv[0].split((Hq, Hkv, Hkv), 1)
        sc.rope(q, k, freqs, lens=s["lens"], slot_ids=slots, D=D, q_out=q, k_out=k)
        sc.pages_append(k, v, s["k"][0], s["v"][0], s["table"], s["lens"], slots, D, **scales(s, 0))
        out = sc.prefix_attention(q, s["k"][0], s["v"][0], s["table"], s["lens"], slots, D, workspace=ws,
                                  **scales(s, 0))
        cu = torch.zeros(6, dtype=torch.int32, device="cuda")
        cu[1:] = s["lens"][slots.long()].cumsum(0)
        k2, v2 = sc.pages_read(s["k"][0], s["v"][0], s["ks"][0], s["vs"][0], s["table"], s["lens"], slots,
                               cu, rows)
        return out, k2, v2

    side = torch.cuda.Stream()
    graphs = []
    for s, qkv, slots, D in cases:
        rows = int(s["lens"].sum())
        fixed = copy_of(s)
        x = qkv.clone()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run(copy_of(s), x.clone(), slots, D)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = run(fixed, x, slots, D)
        graphs.append((graph, fixed, x, got))
    for rep in range(3):
        g = torch.Generator(device="cuda").manual_seed(100 + rep)
        for (graph, fixed, x, got), (s, qkv, slots, D) in zip(graphs, cases):
            rows = int(s["lens"].sum())
            new = torch.randn(qkv.shape, generator=g, device="cuda").bfloat16()
            eager = copy_of(fixed)
            x.copy_(new)
            graph.replay()
            want = run(eager, new.clone(), slots, D)
            torch.cuda.synchronize()
            assert sc.get_error() == 0
            assert all(same(a, b) for a, b in zip(got, want))
            assert all(same(fixed[n], eager[n]) for n in eager)


def test_host_threads_calling_at_once():
    freqs, _ = sc.rope_frequencies(64)
    cases = [prepared(30 + seed) for seed in range(4)]
    want = [step(copy_of(s), qkv.clone(), slots, D, freqs, 1.0) for s, qkv, slots, D in cases]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(j):
        try:
            s, qkv, slots, D = cases[j]
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(8):
                    got[j] = step(copy_of(s), qkv.clone(), slots, D, freqs, 1.0)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # reported on the main thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(j,)) for j in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and sc.get_error() == 0
    for a, b in zip(got, want):
        assert all(same(x, y) for x, y in zip(a, b))


def test_pools_past_two_gigabytes():
    """The last pages of pools of more than 2^31 codes: append, read and attention."""
    ps, Dh, B, heads = 256, 128, 16, 8
    n_pages = (1 << 31) // (ps * heads * Dh) + 40
    k, v, ks, vs = sc.page_cache_8bit(n_pages, ps, heads, Dh, block=B)
    n = 600
    pages = np.array([[n_pages - 1, n_pages - 30, n_pages - 2]])
    table, lens, slots = i32(pages), i32([n]), i32([0])
    g = torch.Generator().manual_seed(1)
    x = torch.randn((n, 2 * heads, Dh), generator=g).bfloat16()
    q = torch.randn((1, 4 * heads, Dh), generator=g).bfloat16()
    sc.pages_append(x[:, :heads].cuda(), x[:, heads:].cuda(), k, v, table, lens, slots, n, k_scales=ks,
                    v_scales=vs)
    got = sc.pages_read(k, v, ks, vs, table, lens, slots, i32([0, n]), n)
    out = sc.prefix_attention(q.cuda(), k, v, table, lens, slots, 1, k_scales=ks, v_scales=vs)
    assert sc.get_error() == 0
    vals = []
    for y, z in ((x[:, :heads], got[0]), (x[:, heads:], got[1])):
        codes, sca = np.zeros((3, ps, heads, Dh), np.uint8), np.ones((3, ps // B, heads), np.float32)
        assert cache8.append(codes, sca, y.double().numpy(), np.array([[0, 1, 2]]), [n], [0], n) == 0
        want = cache8.values(codes, sca)
        vals.append(want)
        assert np.array_equal(z.double().cpu().numpy(), want.reshape(-1, heads, Dh)[:n])
    ref, mag = serving.attention(q.double().numpy(), vals[0], vals[1], np.array([[0, 1, 2]]), [n], [0], 1,
                                 Dh ** -0.5)
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= 1.5 * EPS * mag + 1.01 * EPS * np.abs(ref) + 2.0 ** -40).all()


def test_rope_past_two_to_the_31_values():
    T, heads = (1 << 20) + 3, 32
    q = torch.zeros((T, heads, 64), dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, T // 2, T - 2, T - 1]
    new = torch.randn((5, heads, 64), generator=torch.Generator().manual_seed(2)).bfloat16()
    q[rows] = new.cuda()
    freqs, _ = sc.rope_frequencies(64)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    sc.rope(q, None, freqs, positions=pos, q_out=q)
    few, _ = sc.rope(new.cuda(), None, freqs, positions=i32(rows))
    assert torch.equal(q[rows], few) and sc.get_error() == 0
    q[rows] = 0
    assert not q.any()
