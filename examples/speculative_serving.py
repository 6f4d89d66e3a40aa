"""Speculative serving of a small hybrid decoder: many samples of one prompt.

The decoder alternates ShortConv layers and attention layers over a paged cache. One
prompt is processed once and forked into N branches: their conv states are copied,
their cache pages shared. A step then takes, for every branch, its newest token
and D drafts through all layers at once (conv verify with a window tape, append
to the cache, attention that reads the shared prompt once for all branches),
verifies the drafts against the decoder's probabilities and rolls both kinds of
state back to what was accepted.

    python examples/speculative_serving.py [--branches 16] [--drafts 4] [--steps 20]
                                           [--rotary 64] [--context-factor 4] [--cache-bits 8]

--rotary R turns the first R values of the attention's query and key heads by their positions (as for a
context --context-factor times as long as trained); --cache-bits 8 keeps keys and values as e4m3 codes with a
power of two for every 16 tokens and head.

Weights are random and the draft distribution is the decoder's token-to-token
part, so the figures say how the calls work together, not what a model says.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lfm2_gated_short_gb300 as sc  # noqa: E402


class Decoder:
    """Two ShortConv layers, two attention layers; the residual stream is bf16 [rows, W]."""

    def __init__(self, W=256, V=1000, Hq=8, Hkv=2, Dh=64, K=3, seed=0, rotary=0, context_factor=1.0,
                 cache_bits=16):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape, gain=1.0):
            w = torch.randn(shape, generator=g, device="cuda") * (gain * shape[-1] ** -0.5)
            return w.bfloat16()
        self.W, self.V, self.Hq, self.Hkv, self.Dh, self.K = W, V, Hq, Hkv, Dh, K
        self.cache_bits, self.freqs, self.amplitude = cache_bits, None, 1.0
        if rotary:
            self.freqs, self.amplitude = sc.rope_frequencies(rotary, base=1e6, scaling="parts",
                                                             factor=context_factor)
        self.embed, self.head = weight(V, W, gain=W ** 0.5), weight(V, W, gain=3.0)
        self.conv = [dict(w_in=weight(3 * W, W), w=weight(W, K, gain=1.0), w_out=weight(W, W))
                     for _ in range(2)]
        self.attn = [dict(wqkv=weight((Hq + 2 * Hkv) * Dh, W), w_out=weight(W, Hq * Dh))
                     for _ in range(2)]

    def state(self, n_slots, max_pages, n_pages, page_size):
        """Conv states [layer, slot, W, K], cache tables, and pools [layer, page, token, Hkv, Dh]."""
        refs, table, lens = sc.page_cache(n_slots, max_pages, n_pages)
        bf = dict(dtype=torch.bfloat16, device="cuda")
        s = dict(conv=torch.zeros((len(self.conv), n_slots, self.W, self.K), **bf), refs=refs,
                 table=table, lens=lens)
        if self.cache_bits == 8:
            k, v, k_scales, v_scales = sc.page_cache_8bit(n_pages, page_size, self.Hkv, self.Dh,
                                                          layers=len(self.attn))
            return dict(s, k=k, v=v, k_scales=k_scales, v_scales=v_scales)
        pool = (len(self.attn), n_pages, page_size, self.Hkv, self.Dh)
        return dict(s, k=torch.zeros(pool, **bf), v=torch.zeros(pool, **bf))

    def forward(self, s, slots, tokens, shared_pages=0):
        """Probabilities [N, T, V] after each of tokens [N, T], already counted in s["lens"];
        the conv layers' window tapes [layer, N, T, W, K] (their states are not advanced)."""
        N, T = tokens.shape
        x = self.embed[tokens.flatten().long()]
        tapes = []
        for l, (conv, attn, pool, k, v) in enumerate(zip(self.conv, self.attn, s["conv"], s["k"], s["v"])):
            bcx = (_norm(x) @ conv["w_in"].t()).contiguous()
            tape, y = sc.verify(bcx, conv["w"], slots, pool, T)
            tapes.append(tape)
            x = x + y @ conv["w_out"].t()
            qkv = _norm(x) @ attn["wqkv"].t()
            q, kn, vn = qkv.unflatten(1, (-1, self.Dh)).split((self.Hq, self.Hkv, self.Hkv), 1)
            if self.freqs is not None:  # in place on the projection, at the cache's positions
                sc.rope(q, kn, self.freqs, lens=s["lens"], slot_ids=slots, D=T,
                        amplitude=self.amplitude, q_out=q, k_out=kn)
            sc.pages_append(kn, vn, k, v, s["table"], s["lens"], slots, T, **scales(s, l))
            out = sc.prefix_attention(q, k, v, s["table"], s["lens"], slots, T,
                                      shared_pages=shared_pages, **scales(s, l))
            x = x + out.flatten(1) @ attn["w_out"].t()
        return self.probabilities(x).view(N, T, self.V), torch.stack(tapes)

    def probabilities(self, x):
        return torch.softmax(_norm(x).float() @ self.head.float().t(), -1)

    def draft(self, token, drafts, g):
        """D drafted tokens a branch and their distributions, from the embeddings alone."""
        probs, tokens = [], []
        for _ in range(drafts):
            p = self.probabilities(self.embed[token.long()])
            token = torch.multinomial(p, 1, generator=g)[:, 0].to(torch.int32)
            probs.append(p)
            tokens.append(token)
        return torch.stack(tokens, 1), torch.stack(probs, 1)


def _norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


def scales(s, layer=None):
    """An 8-bit cache's scales (of one layer) as the cache calls take them; nothing for a bf16 one."""
    return {x: s[x] if layer is None else s[x][layer] for x in ("k_scales", "v_scales") if x in s}


def resize(s, slots, new_lens):
    sc.pages_resize(s["refs"], s["table"], s["lens"], slots, new_lens, s["k"], s["v"], **scales(s))


def advance(s, slots, tapes, kept, new_lens):
    """Keep the first `kept` of a step's tokens: conv states from the tape, cache lengths."""
    sc.rollback_layers(tapes, kept, slots, s["conv"])
    resize(s, slots, new_lens)


def generate(model, prompt, branches, drafts, steps, page_size=16, seed=1):
    """(tokens of each branch, accepted counts [steps, N], state, slots)."""
    i32 = dict(dtype=torch.int32, device="cuda")
    N, T = branches, prompt.shape[0]
    longest = T + steps * (drafts + 1) + 1
    max_pages = -(-longest // page_size)
    prompt_pages = -(-T // page_size)
    s = model.state(N + 1, max_pages, prompt_pages + N * (max_pages - T // page_size) + 1, page_size)
    g = torch.Generator(device="cuda").manual_seed(seed)

    # The prompt, once, in slot 0; its last token goes with the first step.
    source = torch.zeros(1, **i32)
    resize(s, source, torch.full((1,), T - 1, **i32))
    _, tapes = model.forward(s, source, prompt[None, :-1])
    advance(s, source, tapes, torch.full((1,), T - 1, **i32), torch.full((1,), T - 1, **i32))

    # The branches: shared pages, copied conv states.
    slots = torch.arange(1, N + 1, **i32)
    sc.pages_fork(s["refs"], s["table"], s["lens"], source.expand(N).contiguous(), slots, s["k"],
                  s["v"], **scales(s))
    for layer in s["conv"]:
        sc.pool_copy(layer, source.expand(N).contiguous(), slots)
    resize(s, source, torch.zeros(1, **i32))  # the prompt's own sequence is no longer needed

    shared = (T - 1) // page_size
    lens = torch.full((N,), T - 1, **i32)
    last = prompt[-1:].expand(N).contiguous()
    sequences = [[] for _ in range(N)]
    counts = []
    for _ in range(steps):
        tokens, q = model.draft(last, drafts, g)
        resize(s, slots, lens + drafts + 1)
        p, tapes = model.forward(s, slots, torch.cat([last[:, None], tokens], 1), shared)
        u = torch.rand((N, drafts + 1), generator=g, device="cuda")
        accepted, out = sc.draft_accept(p, q, tokens, u)
        lens = lens + accepted + 1
        advance(s, slots, tapes, accepted + 1, lens)
        last = out.gather(1, accepted[:, None].long())[:, 0].contiguous()
        counts.append(accepted)
        for seq, row, a in zip(sequences, out.tolist(), accepted.tolist()):
            seq += row[:a + 1]
    error = sc.get_error()
    if error:
        raise RuntimeError(f"device error word {error:#x}")
    return sequences, torch.stack(counts), s, slots


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--branches", type=int, default=16)
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--prompt", type=int, default=500)
    ap.add_argument("--rotary", type=int, default=0)
    ap.add_argument("--context-factor", type=float, default=1.0)
    ap.add_argument("--cache-bits", type=int, default=16, choices=(8, 16))
    a = ap.parse_args()
    model = Decoder(rotary=a.rotary, context_factor=a.context_factor, cache_bits=a.cache_bits)
    g = torch.Generator(device="cuda").manual_seed(2)
    prompt = torch.randint(0, model.V, (a.prompt,), generator=g, device="cuda", dtype=torch.int32)
    sequences, counts, s, _ = generate(model, prompt, a.branches, a.drafts, a.steps)
    n_used = sc.pages_compact(s["refs"], s["table"], s["lens"], s["k"], s["v"], **scales(s))
    print(f"{a.branches} branches of a {a.prompt}-token prompt: {sum(map(len, sequences))} tokens in "
          f"{a.steps} steps, {counts.float().mean():.2f} of {a.drafts} drafts accepted a step; "
          f"{int(n_used)} cache pages in use, compacted")


if __name__ == "__main__":
    main()
