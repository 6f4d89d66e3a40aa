"""Guard bands around every buffer that the 8-bit cache's and the rotary operators write, on ragged
shapes, and exactly sized workspaces (see test_gpu_guard_bands_serving.py). The bounds-checked tests
shorten a record, so that the kernels' own accesses to its end are refused."""
import numpy as np
import pytest
import torch

import lfm2_gated_short_gb300 as sc
from cache8_util import build, codes_from, i32, on_device, same_codes
from oracle import cache8, serving
from test_gpu_guard_bands import Banded

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -8


def banded_codes(a):
    """A Banded's codes as e4m3."""
    b = Banded(a.shape, torch.uint8, torch.from_numpy(a).cuda())
    return b, b.t.view(torch.float8_e4m3fn)


class Cache:
    def __init__(self, n_slots, max_pages, n_pages, ps, L, Hkv, Dh, B, seed):
        self.m = m = cache8.Cache(n_slots, max_pages, n_pages, ps, L, Hkv, Dh, B,
                                  np.random.default_rng(seed))
        pool = (L, n_pages, ps, Hkv, Dh)
        m.k, m.v = m.k.reshape(pool), m.v.reshape(pool)
        self.bands = {}
        self.bands["k"], self.k = banded_codes(m.k)
        self.bands["v"], self.v = banded_codes(m.v)
        tables = zip(("refs", "table", "lens"), sc.page_cache(n_slots, max_pages, n_pages))
        for name, t in (*tables, ("ks", torch.from_numpy(m.ks)), ("vs", torch.from_numpy(m.vs))):
            self.bands[name] = Banded(t.shape, t.dtype, t.cuda())
            setattr(self, name, self.bands[name].t)

    def call(self, f, n, *args, **kw):
        ws = Banded((sc.pages_workspace_bytes(self.refs.shape[0], n),), torch.uint8)
        out = f(self.refs, self.table, self.lens, *args, self.k, self.v, workspace=ws.t, k_scales=self.ks,
                v_scales=self.vs, **kw)
        ws.check("workspace")
        return out

    def check(self):
        m = self.m
        for name, b in self.bands.items():
            b.check(name)
        for name in ("refs", "table", "lens", "ks", "vs"):
            assert np.array_equal(getattr(self, name).cpu().numpy(), getattr(m, name)), name
        for got, want in ((self.k, m.k), (self.v, m.v)):
            assert same_codes(codes_from(got), want)


@pytest.mark.parametrize("n_slots,max_pages,n_pages,ps,L,Hkv,Dh,B", [
    (7, 5, 29, 8, 2, 1, 16, 8), (40, 130, 531, 16, 1, 3, 32, 8), (3, 3, 7, 64, 3, 2, 64, 16)])
def test_pages(n_slots, max_pages, n_pages, ps, L, Hkv, Dh, B):
    r = np.random.default_rng(n_slots)
    p = Cache(n_slots, max_pages, n_pages, ps, L, Hkv, Dh, B, seed=1)
    for _ in range(4):
        slots = r.permutation(n_slots)[:max(1, n_slots // 2)]
        new = r.integers(0, min(max_pages, 2 * n_pages // n_slots) * ps + 1, len(slots))
        p.call(sc.pages_resize, len(slots), i32(slots), i32(new))
        assert sc.get_error() == p.m.resize(slots, new)
        q = r.permutation(n_slots)
        src, dst = np.repeat(q[:1], n_slots - 1), q[1:]
        p.call(sc.pages_fork, len(dst), i32(src), i32(dst))
        assert sc.get_error() == p.m.fork(src, dst)
        p.check()
        n_used = Banded((1,), torch.int32)
        p.call(sc.pages_compact, 0, n_used=n_used.t)
        n_used.check("n_used")
        assert int(n_used.t) == p.m.compact()
        p.check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ps,Hkv,Dh,B", [(8, 3, 16, 8), (32, 1, 80, 16), (64, 4, 64, 64)])
def test_append_and_read(dtype, ps, Hkv, Dh, B):
    p = Cache(5, 6, 14, ps, 1, Hkv, Dh, B, seed=2)
    slots, lens = [3, 1], [ps + 5, 6 * ps]
    p.call(sc.pages_resize, 2, i32(slots), i32(lens))
    p.m.resize(slots, lens)
    D = ps + 3
    x = torch.randn((2 * D, 2 * Hkv, Dh)).to(dtype)
    xd = x.cuda()
    sc.pages_append(xd[:, :Hkv], xd[:, Hkv:], p.k[0], p.v[0], p.table, p.lens, i32(slots), D,
                    k_scales=p.ks[0], v_scales=p.vs[0])
    for codes, scales, y in ((p.m.k, p.m.ks, x[:, :Hkv]), (p.m.v, p.m.vs, x[:, Hkv:])):
        assert cache8.append(codes[0], scales[0], y.double().numpy(), p.m.table, p.m.lens, slots, D) == 0
    assert sc.get_error() == 0
    p.check()
    cu, start = [0, 7, 7 + 5 * ps], [3, ps - 1]
    T = cu[-1]
    k, v = Banded((T, Hkv, Dh), dtype), Banded((T, Hkv, Dh), dtype)
    sc.pages_read(p.k[0], p.v[0], p.ks[0], p.vs[0], p.table, p.lens, i32(slots), i32(cu), T,
                  starts=i32(start), dtype=dtype, k=k.t, v=v.t)
    assert sc.get_error() == 0
    for b, codes, scales in ((k, p.m.k, p.m.ks), (v, p.m.v, p.m.vs)):
        b.check("read")
        vals = cache8.values(codes[0], scales[0])
        want = np.concatenate([vals[p.m.table[s][t // ps], t % ps] for i, s in enumerate(slots)
                               for t in [np.arange(start[i], start[i] + cu[i + 1] - cu[i])]])
        assert np.array_equal(b.t.double().cpu().numpy(), want, equal_nan=True)


def attention(c, trim=None):
    d = on_device(c)
    ps, Hkv, Dh = c["k"].shape[1:]
    out = Banded(c["q"].shape, torch.bfloat16)
    ws = Banded((sc.prefix_attention_8bit_workspace_bytes(c["q"].shape[1], Hkv, Dh, len(c["slots"]), c["D"],
                                                          c["shared"], ps),), torch.uint8)
    torch.cuda.synchronize()
    if trim:
        sc.bounds_trim_next(*trim)
    sc.prefix_attention(d["q"], d["k"], d["v"], d["table"], d["lens"], d["slots"], c["D"],
                        shared_pages=c["shared"], k_scales=d["ks"], v_scales=d["vs"], out=out.t,
                        workspace=ws.t)
    ws.check("workspace")
    out.check("out")
    return out.t.double().cpu().numpy()


@pytest.mark.parametrize("shared,D,G,Hkv,Dh,B", [(0, 1, 1, 1, 64, 8), (0, 3, 7, 2, 64, 16),
                                                 (0, 2, 5, 2, 128, 8), (3, 1, 3, 4, 64, 16),
                                                 (9, 5, 7, 1, 128, 16), (5, 8, 4, 2, 64, 8),
                                                 (4, 1, 128, 1, 64, 16), (0, 4, 4, 4, 128, 8),
                                                 (105, 8, 64, 2, 64, 16)])
def test_attention(shared, D, G, Hkv, Dh, B):
    c = build([shared * 16 + n for n in (9, 33, 200, 16, 70)], shared=shared, B=B, D=D, G=G, Hkv=Hkv,
              Dh=Dh, seed=G)
    k, v = (np.nan_to_num(cache8.values(c[x], c[x + "s"])) for x in "kv")
    ref, mag = serving.attention(c["q"].double().numpy(), k, v, c["table"], c["lens"], c["slots"], D,
                                 Dh ** -0.5)
    got = attention(c)
    assert sc.get_error() == 0
    over = np.abs(got - ref) - (1.5 * EPS * mag + 1.01 * EPS * np.abs(ref) + 2.0 ** -40)
    assert (over <= 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hkv,Dh,R", [(1, 1, 1, 64, 64), (13, 3, 2, 80, 20), (700, 5, 1, 128, 64),
                                           (5, 2, 2, 7, 6)])
def test_rope(dtype, T, Hq, Hkv, Dh, R):
    q, k = torch.randn((T, Hq, Dh), device="cuda").to(dtype), torch.randn((T, Hkv, Dh), device="cuda").to(dtype)
    freqs, _ = sc.rope_frequencies(R)
    pos = i32(np.arange(T))
    want = sc.rope(q, k, freqs, positions=pos)
    qo, ko = Banded((T, Hq, Dh), dtype), Banded((T, Hkv, Dh), dtype)
    sc.rope(q, k, freqs, positions=pos, q_out=qo.t, k_out=ko.t)
    inq, ink = Banded((T, Hq, Dh), dtype, q), Banded((T, Hkv, Dh), dtype, k)
    sc.rope(inq.t, ink.t, freqs, positions=pos, q_out=inq.t, k_out=ink.t)
    for b, w in ((qo, want[0]), (ko, want[1]), (inq, want[0]), (ink, want[1])):
        b.check("rope")
        assert torch.equal(b.t, w)
    assert sc.get_error() == 0


# ------------------------------------------------ the bounds-checked build refuses

def test_a_shortened_scale_array_is_refused():
    if not sc.bounds_checked():
        return  # the standard build has no records
    c = build([64 * 16], seed=5)
    attention(c, trim=(9, c["vs"].nbytes // 2))  # half of V's scales
    assert sc.get_error() & sc.DEV_OUT_OF_BOUNDS
    assert sc.bounds_take_first_bad() != 0


def test_shortened_pools_and_outputs_are_refused():
    if not sc.bounds_checked():
        return  # the standard build has no records
    x = torch.randn((64, 2, 64), device="cuda").bfloat16()
    k, v, ks, vs = sc.page_cache_8bit(4, 16, 2, 64)
    table, lens, slots = i32([[0, 1, 2, 3]]), i32([64]), i32([0])
    torch.cuda.synchronize()
    sc.bounds_trim_next(3, 64)  # V's pool loses its last head
    sc.pages_append(x, x, k, v, table, lens, slots, 64, k_scales=ks, v_scales=vs)
    assert sc.get_error() == sc.DEV_OUT_OF_BOUNDS and sc.bounds_take_first_bad() != 0
    out = [torch.full_like(x, 7.0) for _ in range(2)]
    torch.cuda.synchronize()
    sc.bounds_trim_next(9, 128)  # k loses its last row's last head
    sc.pages_read(k, v, ks, vs, table, lens, slots, i32([0, 64]), 64, k=out[0], v=out[1])
    assert sc.get_error() == sc.DEV_OUT_OF_BOUNDS and sc.bounds_take_first_bad() != 0
    assert (out[0][-1, 1] == 7.0).all() and (out[0][:-1] != 7.0).any()
    freqs, _ = sc.rope_frequencies(64)
    pos = i32(range(64))
    o = torch.full_like(x, 7.0)
    torch.cuda.synchronize()
    sc.bounds_trim_next(6, 128)  # q_out loses its last head
    sc.rope(x, None, freqs, positions=pos, q_out=o)
    assert sc.get_error() == sc.DEV_OUT_OF_BOUNDS and sc.bounds_take_first_bad() != 0
    assert (o[-1, 1] == 7.0).all() and (o[-1, 0] != 7.0).any()
