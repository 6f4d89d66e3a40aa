"""The paged cache on the GPU against its model: tables, counts and page data equal."""
import numpy as np
import pytest
import torch

import lfm2_gated_short_gb300 as sc
from oracle import serving

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def i32(a):
    return torch.as_tensor(np.asarray(a, np.int32)).cuda()


class Pair:
    """A cache on the GPU and its model, filled alike."""

    def __init__(self, n_slots, max_pages, n_pages, ps, L=1, Hkv=2, Dh=8, dtype="bf16", seed=0):
        self.m = serving.Cache(n_slots, max_pages, n_pages, ps, L, Hkv * Dh,
                               np.random.default_rng(seed))
        self.shape = (L, n_pages, ps, Hkv, Dh)
        self.k = torch.from_numpy(self.m.k).to(DT[dtype]).view(self.shape).cuda()
        self.v = torch.from_numpy(self.m.v).to(DT[dtype]).view(self.shape).cuda()
        self.m.k = self.k.double().cpu().numpy().reshape(self.m.k.shape)
        self.m.v = self.v.double().cpu().numpy().reshape(self.m.v.shape)
        self.refs, self.table, self.lens = sc.page_cache(n_slots, max_pages, n_pages)

    def push(self):
        """Copy the model's tables to the GPU."""
        self.refs, self.table, self.lens = i32(self.m.refs), i32(self.m.table), i32(self.m.lens)

    def check(self, err=0):
        assert sc.get_error() == err
        for name in ("refs", "table", "lens"):
            got = getattr(self, name).cpu().numpy()
            assert np.array_equal(got, getattr(self.m, name)), name
        for got, ref in ((self.k, self.m.k), (self.v, self.m.v)):
            assert np.array_equal(got.double().cpu().numpy().reshape(ref.shape), ref)

    def resize(self, slots, new):
        sc.pages_resize(self.refs, self.table, self.lens, i32(slots), i32(new), self.k, self.v)
        self.check(self.m.resize(slots, new))

    def fork(self, src, dst):
        sc.pages_fork(self.refs, self.table, self.lens, i32(src), i32(dst), self.k, self.v)
        self.check(self.m.fork(src, dst))

    def compact(self):
        n = sc.pages_compact(self.refs, self.table, self.lens, self.k, self.v)
        assert int(n) == self.m.compact()
        self.check()


@pytest.mark.parametrize("seed,ps,dtype,L", [(0, 8, "bf16", 1), (1, 16, "f32", 2), (2, 8, "f32", 3),
                                             (3, 32, "bf16", 2)])
def test_random_histories(seed, ps, dtype, L):
    r = np.random.default_rng(seed)
    p = Pair(9, 7, 40, ps, L, dtype=dtype, seed=seed)
    for _ in range(40):
        op = r.integers(4)
        if op <= 1:
            slots = r.permutation(9)[:r.integers(1, 6)]
            p.resize(slots, r.integers(0, 7 * ps + 1, len(slots)))
        elif op == 2:
            q = r.permutation(9)
            n = r.integers(1, 5)
            p.fork(q[r.integers(0, 2, n)], q[2:2 + n])
        else:
            p.compact()


def test_many_sequences_and_pages():
    """More listed sequences and pages than one pass of the scans takes."""
    r = np.random.default_rng(7)
    p = Pair(1500, 5, 5003, 8, Hkv=1, Dh=8)
    p.resize(np.arange(1500), r.integers(0, 25, 1500))
    p.resize(r.permutation(1500)[:1200], r.integers(0, 25, 1200))
    p.compact()
    q = r.permutation(1500)
    p.fork(q[:700], q[700:1400])
    p.resize(q[:1400], r.integers(0, 30, 1400))
    p.compact()


def test_one_source_many_branches_and_truncations_into_shared_pages():
    p = Pair(40, 20, 300, 16, L=2)
    p.resize([3], [16 * 17 + 5])
    p.fork([3] * 30, np.arange(5, 35))
    p.resize(np.arange(5, 35), np.arange(5, 35) * 8 + 1)
    p.resize([3], [33])
    p.resize(np.arange(5, 35), [0] * 30)


def test_two_sequences_leave_one_shared_page_together():
    p = Pair(3, 4, 12, 8)
    p.resize([0], [24])
    p.fork([0], [1])
    p.resize([0, 1], [19, 20])
    p.resize([0, 1], [24, 24])


def test_empty_and_full():
    p = Pair(4, 4, 8, 8)
    p.compact()
    p.resize([0, 1], [32, 32])
    p.resize([2], [1])                # no page left
    p.fork([0], [2])                  # full pages only: none needed
    p.fork([0], [0])                  # a slot is no branch of itself
    p.resize([0, 2], [31, 9])         # shared pages, no page to copy to: nothing changes
    p.resize([1], [0])
    p.resize([0, 2], [31, 9])
    p.compact()


def test_refusals_in_device_data():
    p = Pair(4, 4, 16, 8)
    p.resize([0, 1], [20, 11])
    p.resize([-1, 2, 4], [3, 9, 3])
    p.resize([0, 3], [33, 5])
    p.resize([0, 3], [-1, 6])
    p.fork([0, 9], [2, 3])
    p.m.lens[3] = 99
    p.push()
    p.resize([3, 0], [1, 8])


def test_bad_table_entries_are_skipped():
    p = Pair(3, 4, 16, 8)
    p.resize([0, 1], [24, 16])
    for bad in (16, -7, 2 ** 30):
        p.table[0, 1] = bad
        sc.pages_compact(p.refs, p.table, p.lens, p.k, p.v)
        assert sc.get_error() == sc.DEV_BAD_PAGE
        assert int(p.table[0, 1]) == bad
    before = p.k.clone()
    sc.pages_fork(p.refs, p.table, p.lens, i32([0]), i32([2]), p.k, p.v)
    assert sc.get_error() == sc.DEV_BAD_PAGE
    assert torch.equal(p.k, before)
    sc.pages_resize(p.refs, p.table, p.lens, i32([0]), i32([0]), p.k, p.v)
    assert sc.get_error() == sc.DEV_BAD_PAGE


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1, 3, 20])
def test_append(dtype, D):
    r = np.random.default_rng(D)
    p = Pair(6, 5, 30, 8, L=2, Hkv=3, Dh=16, dtype=dtype, seed=D)
    slots = [4, 0, 2]
    p.resize(slots, [25, 33, 40])
    wide = torch.randn((3 * D, 2, 3, 16), device="cuda").to(DT[dtype])  # k and v as slices of one row
    for layer in range(2):
        sc.pages_append(wide[:, 0], wide[:, 1], p.k[layer], p.v[layer], p.table, p.lens,
                        i32(slots), D)
        flat = wide.double().cpu().numpy().reshape(3 * D, 2, -1)
        p.m.append(layer, flat[:, 0], flat[:, 1], slots, D)
        p.check()


def test_append_refuses_device_data():
    p = Pair(4, 3, 8, 8, Hkv=2, Dh=8)
    p.resize([0, 1], [3, 9])
    k = torch.zeros((8, 2, 8), dtype=torch.bfloat16, device="cuda")
    args = (p.k[0], p.v[0], p.table, p.lens)
    sc.pages_append(k, k, *args, i32([2, 9]), 4)  # an empty sequence and a bad slot
    assert sc.get_error() == sc.DEV_BAD_LENGTH | sc.DEV_BAD_SLOT
    p.check()
    p.table[1, 1] = 8
    sc.pages_append(k[:1], k[:1], *args, i32([1]), 1)
    assert sc.get_error() == sc.DEV_BAD_PAGE
    p.table[1, 1] = int(p.m.table[1, 1])
    p.check()


def test_tables_alone():
    refs, table, lens = sc.page_cache(4, 4, 16)
    none = torch.empty((0, 16, 8, 1, 8), dtype=torch.bfloat16, device="cuda")
    sc.pages_resize(refs, table, lens, i32([1]), i32([13]), none, none)
    sc.pages_fork(refs, table, lens, i32([1]), i32([2]), none, none)
    assert int(sc.pages_compact(refs, table, lens, none, none)) == 3
    assert sc.get_error() == 0
    assert lens.tolist() == [0, 13, 13, 0] and table[2, :3].tolist() == [0, 2, -1]


def test_offsets_past_32_bits():
    """Pools of 5 GB each: the copied and moved pages lie past 2^32 bytes."""
    ps, Hkv, Dh, n_pages = 64, 8, 128, 41000
    k = torch.zeros((n_pages, ps, Hkv, Dh), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    refs, table, lens = sc.page_cache(3, 4, n_pages)
    refs[:40000] = 1                       # others' pages
    sc.pages_resize(refs, table, lens, i32([0]), i32([ps + 7]), k, v)
    new = torch.randn((ps + 7, Hkv, Dh), device="cuda").bfloat16()
    sc.pages_append(new, -new, k, v, table, lens, i32([0]), ps + 7)
    sc.pages_fork(refs, table, lens, i32([0]), i32([1]), k, v)
    assert table[1].tolist() == [40000, 40002, -1, -1]
    assert torch.equal(k[40002, :7], new[ps:]) and torch.equal(v[40002, :7], -new[ps:])
    assert bool((k[40002, 7:] == 0).all())
    refs[:40000] = 0
    assert int(sc.pages_compact(refs, table, lens, k, v)) == 3
    assert sc.get_error() == 0
    assert table[:2].tolist() == [[0, 1, -1, -1], [0, 2, -1, -1]]
    assert torch.equal(k[0], new[:ps]) and torch.equal(k[1, :7], new[ps:])
    assert torch.equal(v[2, :7], -new[ps:])
