"""Refusals of the serving entry points, before any CUDA call."""
import ctypes

import pytest

import lfm2_gated_short_gb300 as sc
from lfm2_gated_short_gb300 import build as sc_build

OK, EINVAL, EUNSUPPORTED = 0, 1, 2
BF16, F32 = 1, 0
BASE = 1 << 40
A, B, C, D_, E, F, G, H, I, J = (BASE + i * (1 << 36) for i in range(10))


@pytest.fixture(scope="module")
def L():
    sc_build.build()
    return sc.lib()


def resize(L, refs=A, n_pages=64, table=B, lens=C, n_slots=8, max_pages=16, ps=16, slots=D_, new=E,
           n=4, layers=2, tok=1024, k=F, v=G, ws=H, wsb=None, fn="resize"):
    need = L.shortconv_pages_workspace_bytes(max(n_pages, 1), max(n, 0))
    f = getattr(L, "shortconv_pages_" + fn)
    return f(refs, n_pages, table, lens, n_slots, max_pages, ps, slots, new, n, layers, tok, k, v,
             ws, need if wsb is None else need + wsb, None)


PAGE_REFUSALS = [
    (dict(n_pages=0), EINVAL), (dict(n_slots=0), EINVAL), (dict(max_pages=0), EINVAL),
    (dict(ps=0), EINVAL), (dict(ps=4), EUNSUPPORTED), (dict(ps=48), EUNSUPPORTED),
    (dict(ps=512), EUNSUPPORTED), (dict(n=-1), EINVAL), (dict(n=9), EINVAL),
    (dict(layers=-1), EINVAL), (dict(tok=0), EINVAL), (dict(tok=24), EUNSUPPORTED),
    (dict(n_slots=1 << 20, max_pages=1 << 12), EUNSUPPORTED), (dict(wsb=-1), EINVAL),
    (dict(refs=0), EINVAL), (dict(refs=A + 2), EINVAL), (dict(table=0), EINVAL),
    (dict(lens=C + 1), EINVAL), (dict(slots=0), EINVAL), (dict(new=E + 2), EINVAL),
    (dict(k=F + 8), EINVAL), (dict(v=0), EINVAL), (dict(ws=H + 4), EINVAL),
    (dict(k=G), EINVAL), (dict(table=A + 16), EINVAL), (dict(lens=B), EINVAL),
    (dict(slots=C), EINVAL), (dict(new=B + 64), EINVAL), (dict(ws=F), EINVAL),
]


@pytest.mark.parametrize("fn", ["resize", "fork"])
@pytest.mark.parametrize("kw,status", PAGE_REFUSALS)
def test_resize_and_fork_refuse(L, fn, kw, status):
    assert resize(L, fn=fn, **kw) == status


@pytest.mark.parametrize("fn", ["resize", "fork"])
def test_nothing_listed_is_ok_without_a_device(L, fn):
    assert resize(L, fn=fn, n=0, slots=0, new=0) == OK


def test_compact_refuses(L):
    def call(k=F, used=E, wsb=0, ps=16, lens=C):
        need = L.shortconv_pages_workspace_bytes(64, 0)
        return L.shortconv_pages_compact(A, 64, B, lens, 8, 16, ps, 1, 1024, k, G, used, H,
                                         need + wsb, None)
    assert call(k=G) == EINVAL
    assert call(used=0) == EINVAL
    assert call(used=A + 4) == EINVAL
    assert call(wsb=-1) == EINVAL
    assert call(ps=24) == EUNSUPPORTED
    assert call(lens=B) == EINVAL


def test_append_refuses(L):
    def call(k=A, ks=1024, v=B, vs=1024, N=4, D=2, tok=1024, kp=C, vp=D_, n_pages=64, ps=16, table=E,
             lens=F, slots=G):
        return L.shortconv_pages_append(k, ks, v, vs, N, D, tok, kp, vp, n_pages, ps, table, lens, 8,
                                        16, slots, None)
    assert call(N=0, k=0, v=0, slots=0) == OK
    for kw, st in [(dict(ks=1008), EINVAL), (dict(vs=1032), EUNSUPPORTED), (dict(D=0), EINVAL),
                   (dict(N=-1), EINVAL), (dict(tok=1000), EUNSUPPORTED), (dict(k=A + 8), EINVAL),
                   (dict(kp=A), EINVAL), (dict(vp=C + 1024), EINVAL), (dict(ps=12), EUNSUPPORTED),
                   (dict(lens=D_), EINVAL), (dict(slots=0), EINVAL)]:
        assert call(**kw) == st, kw


def test_attention_refuses(L):
    def call(dtype=BF16, Hq=32, Hkv=8, Dh=64, q=A, qs=2048, N=4, D=2, kp=B, vp=C, n_pages=64, ps=16,
             table=D_, lens=E, slots=F, shared=0, scale=0.125, out=G, ws=H, wsb=0, max_pages=16):
        need = L.shortconv_prefix_attention_workspace_bytes(32, 8, 64, 4, 2, 0)
        return L.shortconv_prefix_attention(dtype, Hq, Hkv, Dh, q, qs, N, D, kp, vp, n_pages, ps,
                                            table, lens, 8, max_pages, slots, shared, scale, out, ws,
                                            need + wsb, None)
    assert call(N=0, q=0, out=0, slots=0) == OK
    nan = float("nan")
    for kw, st in [(dict(dtype=F32), EUNSUPPORTED), (dict(dtype=9), EUNSUPPORTED),
                   (dict(Hq=30), EINVAL), (dict(Hkv=0), EINVAL), (dict(Dh=96, qs=1 << 12), EUNSUPPORTED),
                   (dict(qs=2040), EINVAL), (dict(qs=2052), EUNSUPPORTED), (dict(D=0), EINVAL),
                   (dict(N=-1), EINVAL), (dict(shared=-1), EINVAL), (dict(shared=17), EINVAL),
                   (dict(scale=0.0), EINVAL), (dict(scale=nan), EINVAL),
                   (dict(scale=float("inf")), EUNSUPPORTED), (dict(ps=20), EUNSUPPORTED),
                   (dict(wsb=-1), EINVAL), (dict(q=0), EINVAL), (dict(out=G + 8), EINVAL),
                   (dict(out=A), EINVAL), (dict(ws=B), EINVAL), (dict(ws=G), EINVAL),
                   (dict(table=0), EINVAL), (dict(lens=E + 2), EINVAL),
                   (dict(Hq=8 * 129, qs=1 << 20), EUNSUPPORTED)]:
        assert call(**kw) == st, kw
    ws = L.shortconv_prefix_attention_workspace_bytes
    assert ws(32, 8, 64, 4, 2, 0) > 0 and ws(32, 8, 64, 4, 2, 0) % 16 == 0
    assert ws(32, 8, 96, 4, 2, 0) == 0 and ws(30, 8, 64, 4, 2, 0) == 0


def test_draft_accept_refuses(L):
    def call(dtype=F32, V=1000, N=4, D=3, t=A, ts=1000, d=B, ds=1000, tok=C, nd=D_, u=E, acc=F, out=G):
        return L.shortconv_draft_accept(dtype, V, N, D, t, ts, d, ds, tok, nd, u, acc, out, None)
    assert call(N=0, t=0, tok=0, u=0, acc=0, out=0) == OK
    for kw, st in [(dict(dtype=5), EUNSUPPORTED), (dict(V=0), EINVAL), (dict(D=-1), EINVAL),
                   (dict(N=-1), EINVAL), (dict(ts=999), EINVAL), (dict(ds=999), EINVAL),
                   (dict(V=(1 << 22) + 1, ts=1 << 23, ds=1 << 23), EUNSUPPORTED), (dict(t=0), EINVAL),
                   (dict(t=A + 2), EINVAL), (dict(tok=0), EINVAL), (dict(u=0), EINVAL),
                   (dict(acc=F + 2), EINVAL), (dict(out=A + 64), EINVAL), (dict(acc=G), EINVAL),
                   (dict(out=E), EINVAL), (dict(nd=D_ + 1), EINVAL)]:
        assert call(**kw) == st, kw


def test_binding_refuses_what_the_library_cannot_see():
    torch = pytest.importorskip("torch")
    t = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError):  # host tensors
        sc.draft_accept(t, t[:, :2], torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 3))
    with pytest.raises(ValueError):  # rows not contiguous
        sc._rows(torch.zeros(4, 6).t(), "x", torch.float32, (6, 4))
