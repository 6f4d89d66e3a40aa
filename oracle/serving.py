"""Plain definitions of the speculative serving operators -- TEST INFRASTRUCTURE.

Numpy, in float64 and whole numbers, one loop a definition: the paged cache's
resize, fork, compaction and append (in place on numpy arrays), the attention of
a step over it, and the verification of drafted tokens. Only tests may import this
module, like the rest of ``oracle/``.
"""
from __future__ import annotations

import numpy as np

NO_PAGE, BAD_PAGE, BAD_LENGTH, BAD_TOKEN, BAD_PROBS = 0x40, 0x80, 0x100, 0x200, 0x400
BAD_SLOT, BAD_ACCEPTED = 0x1, 0x4


class Cache:
    """refs, table, lens and pools ``[L, n_pages, page_size, width]``; every method returns
    the error bits it would set."""

    def __init__(self, n_slots, max_pages, n_pages, page_size, L=1, width=8, rng=None):
        self.ps, self.n_pages = page_size, n_pages
        self.refs = np.zeros(n_pages, np.int64)
        self.table = np.full((n_slots, max_pages), -1, np.int64)
        self.lens = np.zeros(n_slots, np.int64)
        shape = (L, n_pages, page_size, width)
        rng = rng or np.random.default_rng(0)
        self.k, self.v = rng.standard_normal(shape), rng.standard_normal(shape)

    def pages(self, n):
        return -(-int(n) // self.ps)

    def _length_error(self, slot):
        if not 0 <= slot < len(self.lens):
            return BAD_SLOT
        return 0 if 0 <= self.lens[slot] <= self.table.shape[1] * self.ps else BAD_LENGTH

    def _copy(self, src, dst, rows):
        self.k[:, dst, :rows] = self.k[:, src, :rows]
        self.v[:, dst, :rows] = self.v[:, src, :rows]

    def resize(self, slots, new_lens):
        err, todo = 0, []
        for s, n in zip(slots, new_lens):
            e = self._length_error(s)
            if not e and not 0 <= n <= self.table.shape[1] * self.ps:
                e = BAD_LENGTH
            err |= e
            if not e:
                todo.append((int(s), int(n)))
        refs = self.refs.copy()
        for s, n in todo:
            for e in range(self.pages(n), self.pages(self.lens[s])):
                refs[self.table[s, e]] -= 1
        plan, want = [], 0
        for s, n in todo:
            need, have = self.pages(n), self.pages(self.lens[s])
            copy = n < self.lens[s] and n % self.ps != 0 and refs[self.table[s, need - 1]] > 1
            plan.append((s, n, need, have, copy))
            want += int(copy) + max(0, need - have)
        free = list(np.nonzero(refs == 0)[0])
        if len(free) < want:
            return err | NO_PAGE
        self.refs = refs
        copies = []
        for s, n, need, have, copy in plan:
            self.table[s, need:have] = -1
            if copy:
                old, new = self.table[s, need - 1], free.pop(0)
                self.refs[old] -= 1
                self.refs[new] = 1
                self.table[s, need - 1] = new
                copies.append((old, new, n % self.ps))
            for e in range(have, need):
                self.table[s, e] = free.pop(0)
                self.refs[self.table[s, e]] = 1
            self.lens[s] = n
        for c in copies:
            self._copy(*c)
        return err

    def fork(self, src, dst):
        err, todo = 0, []
        for s, d in zip(src, dst):
            e = self._length_error(s) | self._length_error(d)
            if not e and s == d:
                e = BAD_SLOT
            err |= e
            if not e:
                todo.append((int(s), int(d)))
        refs = self.refs.copy()
        for _, d in todo:
            for e in range(self.pages(self.lens[d])):
                refs[self.table[d, e]] -= 1
        free = list(np.nonzero(refs == 0)[0])
        if len(free) < sum(self.lens[s] % self.ps != 0 for s, _ in todo):
            return err | NO_PAGE
        self.refs = refs
        for s, d in todo:
            full, part = divmod(int(self.lens[s]), self.ps)
            row = np.full_like(self.table[d], -1)
            row[:full] = self.table[s, :full]
            self.refs[row[:full]] += 1
            if part:
                row[full] = free.pop(0)
                self.refs[row[full]] = 1
                self._copy(self.table[s, full], row[full], part)
            self.table[d], self.lens[d] = row, self.lens[s]
        return err

    def compact(self):
        used = int((self.refs > 0).sum())
        movers = [p for p in range(used, self.n_pages) if self.refs[p] > 0]
        holes = [p for p in range(used) if self.refs[p] == 0]
        for src, dst in zip(movers, holes):
            self._copy(src, dst, self.ps)
            self.refs[dst], self.refs[src] = self.refs[src], 0
            self.table[self.table == src] = dst
        return used

    def append(self, layer, k, v, slots, D):
        for i, s in enumerate(slots):
            for j in range(D):
                pos = int(self.lens[s]) - D + j
                page = self.table[s, pos // self.ps]
                self.k[layer, page, pos % self.ps] = k[i * D + j]
                self.v[layer, page, pos % self.ps] = v[i * D + j]


def attention(q, k_pages, v_pages, table, lens, slots, D, scale):
    """``(out, mean |v|)`` of ``q [N*D, Hq, Dh]`` over ``[n_pages, ps, Hkv, Dh]`` pages, float64:
    the weighted mean of the visible values, and of their magnitudes (for error bounds)."""
    q, k_pages, v_pages = (np.asarray(x, np.float64) for x in (q, k_pages, v_pages))
    _, Hq, Dh = q.shape
    ps, Hkv = k_pages.shape[1], k_pages.shape[2]
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    for i, s in enumerate(slots):
        for j in range(D):
            n = int(lens[s]) - D + j + 1
            if n <= 0:
                continue
            t = np.arange(n)
            keys = k_pages[table[s][t // ps], t % ps]
            vals = v_pages[table[s][t // ps], t % ps]
            for h in range(Hq):
                z = scale * (keys[:, h // (Hq // Hkv)] @ q[i * D + j, h])
                w = np.exp(z - z.max())
                w /= w.sum()
                out[i * D + j, h] = w @ vals[:, h // (Hq // Hkv)]
                mag[i * D + j, h] = w @ np.abs(vals[:, h // (Hq // Hkv)])
    return out, mag


def _weights(row):
    p = np.nan_to_num(np.asarray(row, np.float64), nan=0.0, posinf=1.0, neginf=0.0)
    return [int(x) for x in np.clip(p, 0.0, 1.0) * 2.0 ** 40]


def draft_accept(target, draft, tokens, uniforms, n_drafts=None):
    """``(errors, accepted [N], out_tokens [N, D+1])`` in whole numbers of any size."""
    N, D1, V = target.shape
    D, err = D1 - 1, 0
    accepted, out = np.zeros(N, np.int64), np.full((N, D1), -1, np.int64)
    for i in range(N):
        n = D if n_drafts is None else int(n_drafts[i])
        if not 0 <= n <= D:
            err |= BAD_ACCEPTED
            continue
        if any(not 0 <= int(x) < V for x in tokens[i, :n]):
            err |= BAD_TOKEN
            continue
        a = 0
        while a < n:
            x = int(tokens[i, a])
            q = 1.0 if draft is None else float(draft[i, a, x])
            if not float(uniforms[i, a]) * q < float(target[i, a, x]):
                break
            a += 1
        w = _weights(target[i, a])
        if a < n:
            if draft is None:
                q = [0] * V
                q[int(tokens[i, a])] = 1 << 40
            else:
                q = _weights(draft[i, a])
            rest = [max(x - y, 0) for x, y in zip(w, q)]
            w = rest if any(rest) else w
        accepted[i], out[i, :a] = a, tokens[i, :a]
        total, mark = sum(w), 0
        mark = total * int(float(uniforms[i, D]) * 2 ** 31) >> 31
        if total == 0:
            err |= BAD_PROBS
            continue
        acc = 0
        for t, x in enumerate(w):
            acc += x
            if acc > mark:
                out[i, a] = t
                break
    return err, accepted, out
