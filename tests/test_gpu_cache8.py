"""The 8-bit cache's append, read, resize, fork and compaction on the GPU against the plain definitions,
bit for bit: a scale is a power of two, so that codes and values have no rounding but the code's own."""
import numpy as np
import pytest
import torch

import lfm2_gated_short_gb300 as sc
from cache8_util import codes_from, codes_to, i32, same_codes
from oracle import cache8

pytestmark = pytest.mark.gpu


def numbers(r, shape, dtype):
    """Rows of unlike sizes, with a few zeros, infinities and NaN; as the tensor's dtype holds them."""
    x = r.standard_normal(shape) * np.exp2(r.integers(-6, 7, shape[:1] + (1,) * (len(shape) - 1)))
    x[r.random(shape) < 0.02] = 0.0
    x[r.random(shape) < 0.002] = np.inf
    x[r.random(shape) < 0.002] = np.nan
    x[r.random(shape[0]) < 0.1] = 0.0
    return torch.from_numpy(x).to(dtype)


class Pair:
    """A model and its tensors, one layer."""

    def __init__(self, n_slots, max_pages, n_pages, ps, Hkv, Dh, B, seed, L=1):
        self.m = cache8.Cache(n_slots, max_pages, n_pages, ps, L, Hkv, Dh, B, np.random.default_rng(seed))
        m, pool = self.m, (L, n_pages, ps, Hkv, Dh)
        self.k, self.v = codes_to(m.k).view(pool), codes_to(m.v).view(pool)
        self.ks, self.vs = torch.from_numpy(m.ks).cuda(), torch.from_numpy(m.vs).cuda()
        self.refs, self.table, self.lens = sc.page_cache(n_slots, max_pages, n_pages)
        self.pool = pool

    def args(self):
        return dict(k_scales=self.ks, v_scales=self.vs)

    def resize(self, slots, lens):
        err = self.m.resize(slots, lens)
        sc.pages_resize(self.refs, self.table, self.lens, i32(slots), i32(lens), self.k, self.v,
                        **self.args())
        assert sc.get_error() == err
        return err

    def append(self, k, v, slots, D, layer=0, stream=None):
        m, rows = self.m, (-1,) + self.pool[3:]
        err = 0
        for x, codes, scales in ((k, m.k, m.ks), (v, m.v, m.vs)):
            err |= cache8.append(codes[layer].reshape(self.pool[1:]), scales[layer],
                                 x.double().numpy().reshape(rows), m.table, m.lens, slots, D)
        sc.pages_append(k.cuda(), v.cuda(), self.k[layer], self.v[layer], self.table, self.lens,
                        i32(slots), D, stream=stream, k_scales=self.ks[layer], v_scales=self.vs[layer])
        assert sc.get_error() == err

    def check(self):
        m = self.m
        assert np.array_equal(self.table.cpu().numpy(), m.table)
        assert np.array_equal(self.lens.cpu().numpy(), m.lens)
        assert np.array_equal(self.refs.cpu().numpy(), m.refs)
        for got, want in ((self.k, m.k), (self.v, m.v)):
            assert same_codes(codes_from(got).reshape(want.shape), want)
        for got, want in ((self.ks, m.ks), (self.vs, m.vs)):
            assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ps,B,Hkv,Dh", [(8, 8, 1, 64), (16, 8, 2, 64), (16, 16, 8, 64), (32, 16, 3, 128),
                                         (64, 64, 2, 16), (256, 128, 1, 80), (256, 256, 2, 64)])
def test_appends_one_after_the_other(dtype, ps, B, Hkv, Dh):
    """A token, drafts, prompts, rollbacks into blocks and an empty sequence: the whole pools."""
    r = np.random.default_rng(B + Dh)
    N, p = 3, Pair(5, 12 + 640 // ps, 3 * (12 + 640 // ps), ps, Hkv, Dh, B, seed=B)
    slots = [4, 0, 2]
    for grow, keep in ((1, 0), (1, 0), (3, 2), (B, 0), (B + 1, 1), (2 * B + 5, B), (7, 6), (1, 0)):
        p.resize(slots, p.m.lens[slots] + grow)
        p.append(*(numbers(r, (N * grow, Hkv, Dh), dtype) for _ in range(2)), slots, grow)
        p.check()
        if keep:
            p.resize(slots, p.m.lens[slots] - grow + np.minimum(grow, [keep, 0, keep]))
    p.check()


def test_append_from_strided_rows():
    r = np.random.default_rng(5)
    p = Pair(3, 4, 9, 16, 2, 64, 16, seed=5)
    p.resize([1, 2], [40, 23])
    qkv = numbers(r, (2 * 20, 6, 64), torch.bfloat16).cuda()
    p.append(qkv[:, 2:4].cpu(), qkv[:, 4:].cpu(), [1, 2], 20)
    before = [x.clone() for x in (p.k, p.ks)]
    sc.pages_append(qkv[:, 2:4], qkv[:, 4:], p.k[0], p.v[0], p.table, p.lens, i32([1, 2]), 20,
                    k_scales=p.ks[0], v_scales=p.vs[0])
    p.check()
    assert torch.equal(before[0].view(torch.uint8), p.k.view(torch.uint8))  # a second time: the same
    assert torch.equal(before[1], p.ks)


def test_append_sizes_at_the_ends_of_the_range():
    p = Pair(2, 2, 3, 8, 1, 16, 8, seed=6)
    for rows in ([3.3e38, -3e38], [1e-30, 2e-38], [448.0, 449.0, 224.0], [0.0], [float("inf")],
                 [float("nan"), 3.0], [2.0 ** -64 * 448, 2.0 ** -75]):
        x = torch.zeros((1, 1, 16))
        x[0, 0, :len(rows)] = torch.tensor(rows)
        for first in (1, 0):  # behind an earlier token, and the block's first
            p.resize([1], [0])
            p.resize([1], [1 + first])
            if first:
                p.append(torch.ones((2, 1, 16)) * 0.3, torch.ones((2, 1, 16)) * 1e5, [1], 2)
            p.append(x, -x, [1], 1)
            p.check()


def test_scales_that_hold_anything_before_the_first_append():
    p = Pair(2, 2, 3, 8, 1, 16, 8, seed=7)
    p.ks.fill_(float("nan"))
    p.vs.fill_(-float("inf"))
    p.m.ks[:], p.m.vs[:] = np.nan, -np.inf
    p.resize([0], [3])
    x = numbers(np.random.default_rng(7), (3, 1, 16), torch.float32)
    p.append(x, x, [0], 3)
    assert np.array_equal(p.ks.cpu().numpy(), p.m.ks, equal_nan=True)
    assert same_codes(codes_from(p.k).reshape(p.m.k.shape), p.m.k)


def test_append_with_bad_slots_lengths_and_pages():
    r = np.random.default_rng(8)
    p = Pair(6, 4, 20, 16, 2, 64, 8, seed=8)
    p.resize([0, 1, 2, 3], [20, 30, 2, 33])
    p.m.table[1, 1] = p.m.n_pages
    p.m.lens[3] = 65
    p.table.copy_(i32(p.m.table))
    p.lens.copy_(i32(p.m.lens))
    x = numbers(r, (6 * 5, 2, 64), torch.bfloat16)
    p.append(x, x, [0, 1, 2, 3, 6, -1], 5)  # sound, bad page, shorter than D, too long, no slots
    for got, want in ((p.k, p.m.k), (p.v, p.m.v)):
        assert same_codes(codes_from(got).reshape(want.shape), want)
    assert np.array_equal(p.ks.cpu().numpy(), p.m.ks)


@pytest.mark.parametrize("L,Hkv,Dh,ps,B", [(2, 1, 64, 16, 8), (3, 8, 64, 16, 16), (1, 3, 16, 32, 8)])
def test_forks_rollbacks_and_compactions_take_the_scales_along(L, Hkv, Dh, ps, B):
    r = np.random.default_rng(9)
    p = Pair(40, 20, 300, ps, Hkv, Dh, B, seed=9, L=L)
    n = 5 * ps + 3
    p.resize([0, 1], [n, 2 * ps])
    for layer in range(L):
        p.append(*(numbers(r, (n, Hkv, Dh), torch.bfloat16) for _ in range(2)), [0], n, layer)
    dst = list(range(2, 36))
    assert p.m.fork([0] * 34, dst) == 0
    sc.pages_fork(p.refs, p.table, p.lens, i32([0] * 34), i32(dst), p.k, p.v, **p.args())
    p.check()
    p.resize(dst[:3], [2 * ps + 5, 2 * ps + 1, n])  # into pages that others share
    p.resize(dst[:3], [2 * ps + 6, 2 * ps + 2, n + 1])
    for layer in range(L):
        p.append(*(numbers(r, (3, Hkv, Dh), torch.bfloat16) for _ in range(2)), dst[:3], 1, layer)
    p.check()
    p.resize(dst[3:30] + [1], [0] * 28)
    used = sc.pages_compact(p.refs, p.table, p.lens, p.k, p.v, **p.args())
    assert int(used) == p.m.compact()
    p.check()
    assert sc.get_error() == 0


def test_one_large_copy_list_takes_its_own_kernel():
    """More bytes than the table kernels copy themselves."""
    p = Pair(70, 3, 300, 256, 8, 64, 16, seed=10)
    p.resize([0], [300])
    assert p.m.fork([0] * 60, range(1, 61)) == 0
    sc.pages_fork(p.refs, p.table, p.lens, i32([0] * 60), i32(range(1, 61)), p.k, p.v, **p.args())
    p.check()


def filled(N, ps, Hkv, Dh, B, seed, lens):
    p = Pair(N + 2, max(1, -(-max(lens) // ps)), sum(-(-n // ps) for n in lens) + 3, ps, Hkv, Dh, B, seed)
    slots = np.random.default_rng(seed).permutation(N + 2)[:N]
    p.resize(slots, lens)
    return p, slots


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ps,B,Hkv,Dh", [(8, 8, 1, 16), (16, 8, 2, 64), (64, 16, 8, 64), (32, 32, 3, 128)])
@pytest.mark.parametrize("starts", [False, True])
def test_read(dtype, ps, B, Hkv, Dh, starts):
    lens = [1, 0, 7, 8, 130, 33, 300]
    p, slots = filled(7, ps, Hkv, Dh, B, 11, lens)
    r = np.random.default_rng(11)
    start = np.array([r.integers(0, n + 1) for n in lens]) if starts else np.zeros(7, int)
    count = np.array([r.integers(0, n - s + 1) if starts else n for n, s in zip(lens, start)])
    cu = np.concatenate([[0], np.cumsum(count)])
    k, v = sc.pages_read(p.k[0], p.v[0], p.ks[0], p.vs[0], p.table, p.lens, i32(slots), i32(cu),
                         int(cu[-1]), starts=i32(start) if starts else None, dtype=dtype)
    assert sc.get_error() == 0 and k.dtype == dtype
    for got, codes, scales in ((k, p.m.k[0], p.m.ks[0]), (v, p.m.v[0], p.m.vs[0])):
        x = cache8.values(codes.reshape(p.pool[1:]), scales)
        want = [x[p.m.table[s][t // ps], t % ps] for i, s in enumerate(slots)
                for t in [np.arange(start[i], start[i] + count[i])]]
        want = np.concatenate(want)
        assert np.array_equal(got.double().cpu().numpy(), want, equal_nan=True)


def test_read_leaves_bad_sequences_rows_alone():
    p, slots = filled(5, 16, 2, 64, 8, 12, [20, 20, 20, 20, 20])
    s = list(slots)
    p.m.lens[s[1]] = 999
    p.m.table[s[2], 1] = -1
    p.lens.copy_(i32(p.m.lens))
    p.table.copy_(i32(p.m.table))
    listed = [s[0], s[1], s[2], -3, s[4], s[0]]  # a slot twice
    cu, start = [0, 20, 25, 45, 50, 70, 73], [0, 0, 0, 0, 1, 17]  # 1 + 20 tokens of 20
    out = [torch.full((73 + 5, 2, 64), 5.0, device="cuda") for _ in range(2)]
    sc.pages_read(p.k[0], p.v[0], p.ks[0], p.vs[0], p.table, p.lens, i32(listed), i32(cu), 73,
                  starts=i32(start), dtype=torch.float32, k=out[0][:73], v=out[1][:73])
    assert sc.get_error() == sc.DEV_BAD_SLOT | sc.DEV_BAD_LENGTH | sc.DEV_BAD_PAGE
    for got, codes, scales in ((out[0], p.m.k[0], p.m.ks[0]), (out[1], p.m.v[0], p.m.vs[0])):
        x = cache8.values(codes.reshape(p.pool[1:]), scales)
        got, want = got.double().cpu().numpy(), np.full((78, 2, 64), 5.0)
        row = p.m.table[s[0]]
        want[:20] = x[row[np.arange(20) // 16], np.arange(20) % 16]
        want[25:41] = x[p.m.table[s[2], 0]]  # the page before the bad one
        t = np.arange(17, 20)
        want[70:73] = x[row[t // 16], t % 16]
        assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("cu", [[1, 5, 9], [0, 6, 5], [0, 5, 8], [0, 5, 10], [0, -1, 9]])
def test_read_refuses_bad_seqlens_whole(cu):
    p, slots = filled(2, 16, 1, 16, 8, 13, [10, 10])
    out = [torch.full((9, 1, 16), 5.0, device="cuda") for _ in range(2)]
    sc.pages_read(p.k[0], p.v[0], p.ks[0], p.vs[0], p.table, p.lens, i32(slots), i32(cu), 9,
                  dtype=torch.float32, k=out[0], v=out[1])
    assert sc.get_error() == sc.DEV_BAD_SEQLENS
    assert (out[0] == 5.0).all() and (out[1] == 5.0).all()


def test_read_of_many_rows():
    """More tiles than CTAs."""
    p, slots = filled(3, 256, 1, 16, 32, 14, [30000, 1, 30001])
    cu = np.array([0, 30000, 30001, 60002])
    k, _ = sc.pages_read(p.k[0], p.v[0], p.ks[0], p.vs[0], p.table, p.lens, i32(slots), i32(cu), 60002,
                         dtype=torch.float32)
    x = cache8.values(p.m.k[0].reshape(p.pool[1:]), p.m.ks[0])
    want = np.concatenate([x[p.m.table[s][t // 256], t % 256] for s, n in zip(slots, (30000, 1, 30001))
                           for t in [np.arange(n)]])
    assert np.array_equal(k.double().cpu().numpy(), want, equal_nan=True)
