"""The serving operators on several streams, in CUDA graphs and from several host threads."""
import threading

import numpy as np
import pytest
import torch

import lfm2_gated_short_gb300 as sc
from test_gpu_draft_accept import inputs
from test_gpu_pages import i32
from test_gpu_prefix_attention import build

pytestmark = pytest.mark.gpu


def step_args(seed, shared=6, N=12, D=3):
    r = np.random.default_rng(seed)
    c = build(r.integers(shared * 16 + 20, shared * 16 + 600, N), shared=shared, D=D, G=4, seed=seed)
    c["lens"][c["slots"]] = np.maximum(c["lens"][c["slots"]], D)
    dev = dict(q=c["q"].cuda(), k=c["k"].cuda(), v=c["v"].cuda(), table=i32(c["table"]),
               lens=i32(c["lens"]), slots=i32(c["slots"]))
    g = torch.Generator().manual_seed(seed)
    dev["kn"] = torch.randn((N * D, 2, 64), generator=g).bfloat16().cuda()
    return dev, shared, D


def step(a, shared, D, stream=None, out=None):
    sc.pages_append(a["kn"], -a["kn"], a["k"], a["v"], a["table"], a["lens"], a["slots"], D,
                    stream=stream)
    return sc.prefix_attention(a["q"], a["k"], a["v"], a["table"], a["lens"], a["slots"], D,
                               shared_pages=shared, out=out, stream=stream)


def test_interleaved_on_streams_given_and_current():
    cases = [step_args(s, shared) for s, shared in ((1, 6), (2, 0), (3, 40), (4, 3))]
    ref = [step(*c).clone() for c in cases]
    probs = inputs(6, 4, 5000, "f32", seed=5)
    probs = [t.cuda() for t in probs]
    ref_tokens = sc.draft_accept(*probs)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.empty_like(r) for r in ref]
    torch.cuda.synchronize()
    tokens = []
    for rep in range(8):
        for c, st, out in zip(cases, streams, outs):
            if rep % 2:
                step(*c, stream=st, out=out)  # the call's workspace belongs to `st`
            else:
                with torch.cuda.stream(st):
                    step(*c, out=out)
            with torch.cuda.stream(st):
                tokens.append(sc.draft_accept(*probs))
    torch.cuda.synchronize()
    assert sc.get_error() == 0
    for out, r in zip(outs, ref):
        assert torch.equal(out, r)
    for a, t in tokens:
        assert torch.equal(a, ref_tokens[0]) and torch.equal(t, ref_tokens[1])


def test_a_captured_serving_step():
    """Resize, append, attention and acceptance replayed from a graph, on new inputs each time."""
    N, D, V, ps, Hkv, Dh = 5, 3, 700, 16, 2, 64
    r = np.random.default_rng(7)

    def state():
        refs, table, lens = sc.page_cache(N + 1, 20, 130)
        k = torch.zeros((130, ps, Hkv, Dh), dtype=torch.bfloat16, device="cuda")
        v = torch.zeros_like(k)
        slots = i32(np.arange(1, N + 1))
        sc.pages_resize(refs, table, lens, i32([0]), i32([100]), k, v)
        new = torch.from_numpy(r.standard_normal((100, Hkv, Dh))).bfloat16().cuda()
        sc.pages_append(new, -new, k, v, table, lens, i32([0]), 100)
        sc.pages_fork(refs, table, lens, i32([0] * N), slots, k, v)
        return dict(refs=refs, table=table, lens=lens, k=k, v=v, slots=slots)

    def run(s, x):
        room = s["lens"][1:] + D
        sc.pages_resize(s["refs"], s["table"], s["lens"], s["slots"], room, s["k"], s["v"])
        sc.pages_append(x["kn"], x["kn"], s["k"], s["v"], s["table"], s["lens"], s["slots"], D)
        out = sc.prefix_attention(x["q"], s["k"], s["v"], s["table"], s["lens"], s["slots"], D,
                                  shared_pages=6)
        a, t = sc.draft_accept(x["p"], None, x["tokens"], x["u"])
        sc.pages_resize(s["refs"], s["table"], s["lens"], s["slots"], room - D + a, s["k"], s["v"])
        return out, a, t

    def new_inputs(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        p = torch.softmax(torch.randn((N, D + 1, V), generator=g, device="cuda") * 3, -1)
        q = torch.randn((N * D, 4, Dh), generator=g, device="cuda").bfloat16()
        kn = torch.randn((N * D, Hkv, Dh), generator=g, device="cuda").bfloat16()
        return dict(p=p, q=q, kn=kn, tokens=p[:, :D].argmax(-1).to(torch.int32),
                    u=torch.rand((N, D + 1), generator=g, device="cuda"))
    r = np.random.default_rng(7)
    eager = state()
    r = np.random.default_rng(7)
    graphed = state()
    x = new_inputs(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # warm up on a throwaway state
        run(state(), x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = run(graphed, x)
    for seed in range(1, 6):
        for name, t in new_inputs(seed).items():
            x[name].copy_(t)
        graph.replay()
        ref = run(eager, x)
        torch.cuda.synchronize()
        assert sc.get_error() == 0
        for g_, r_ in zip(got, ref):
            assert torch.equal(g_, r_)
        for name in ("refs", "table", "lens", "k", "v"):
            assert torch.equal(graphed[name], eager[name]), name


def test_host_threads_calling_at_once():
    cases = [step_args(10 + s, shared) for s, shared in enumerate((6, 0, 30, 2))]
    ref = [step(*c).clone() for c in cases]
    torch.cuda.synchronize()
    got, errors = [None] * len(cases), []

    def work(j):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(15):
                    got[j] = step(*cases[j])
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # reported on the main thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(j,)) for j in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    assert sc.get_error() == 0
    for g_, r_ in zip(got, ref):
        assert torch.equal(g_, r_)
