"""Refusals of the 8-bit cache's and the rotary entry points, before any CUDA call."""
import ctypes

import pytest

import lfm2_gated_short_gb300 as sc
from lfm2_gated_short_gb300 import build as sc_build

OK, EINVAL, EUNSUPPORTED = 0, 1, 2
BF16, F32 = 1, 0
BASE = 1 << 40
A, B, C, D_, E, F, G, H, I, J, K_ = (BASE + i * (1 << 36) for i in range(11))


@pytest.fixture(scope="module")
def L():
    sc_build.build()
    return sc.lib()


def append(L, dt=BF16, Hkv=2, Dh=64, block=16, k=A, ks=256, v=B, vs=256, N=3, D=2, kp=C, vp=D_, kc=E,
           vc=F, n_pages=64, ps=32, table=G, lens=H, n_slots=8, max_pages=16, slots=I):
    return L.shortconv_pages_append_8bit(dt, Hkv, Dh, block, k, ks, v, vs, N, D, kp, vp, kc, vc, n_pages,
                                         ps, table, lens, n_slots, max_pages, slots, None)


SHAPES = [(dict(Hkv=0), EINVAL), (dict(Dh=0), EINVAL), (dict(Dh=24), EUNSUPPORTED),
          (dict(block=0), EINVAL), (dict(block=4), EUNSUPPORTED), (dict(block=24), EUNSUPPORTED),
          (dict(block=64), EUNSUPPORTED), (dict(ps=48), EUNSUPPORTED), (dict(ps=4), EUNSUPPORTED),
          (dict(n_pages=0), EINVAL), (dict(n_slots=0), EINVAL), (dict(max_pages=0), EINVAL)]


@pytest.mark.parametrize("kw,status", SHAPES + [
    (dict(dt=7), EUNSUPPORTED), (dict(N=-1), EINVAL), (dict(D=0), EINVAL), (dict(ks=64), EINVAL),
    (dict(vs=129), EUNSUPPORTED), (dict(dt=F32, vs=130), EUNSUPPORTED), (dict(k=A + 8), EINVAL),
    (dict(v=0), EINVAL), (dict(kp=0), EINVAL), (dict(vp=D_ + 4), EINVAL), (dict(kc=E + 2), EINVAL),
    (dict(vc=0), EINVAL), (dict(table=0), EINVAL), (dict(lens=H + 1), EINVAL), (dict(slots=0), EINVAL),
    (dict(vp=C), EINVAL), (dict(kc=C + 64), EINVAL), (dict(vc=E), EINVAL), (dict(k=C), EINVAL),
    (dict(table=F), EINVAL), (dict(N=1 << 20, D=1 << 12), EINVAL),
    (dict(N=1 << 28, D=1, Hkv=1 << 10, Dh=16, ks=1 << 14, vs=1 << 14), EINVAL),
    (dict(ks=1 << 37), EUNSUPPORTED)])
def test_append_refuses(L, kw, status):
    assert append(L, **kw) == status


def test_nothing_to_append_is_ok_without_a_device(L):
    assert append(L, N=0, k=0, v=0, slots=0) == OK


def read(L, dt=BF16, Hkv=2, Dh=64, block=16, kp=A, vp=B, kc=C, vc=D_, n_pages=64, ps=32, table=E, lens=F,
         n_slots=8, max_pages=16, slots=G, cu=H, starts=0, N=3, T=50, k=I, v=J):
    return L.shortconv_pages_read_8bit(dt, Hkv, Dh, block, kp, vp, kc, vc, n_pages, ps, table, lens,
                                       n_slots, max_pages, slots, cu, starts or None, N, T, k, v, None)


@pytest.mark.parametrize("kw,status", SHAPES + [
    (dict(dt=3), EUNSUPPORTED), (dict(N=-1), EINVAL), (dict(T=-1), EINVAL), (dict(T=1 << 31), EINVAL),
    (dict(N=0, slots=0, T=1), EINVAL), (dict(kp=A + 4), EINVAL), (dict(vc=0), EINVAL), (dict(cu=0), EINVAL),
    (dict(slots=0), EINVAL), (dict(starts=K_ + 2), EINVAL), (dict(k=0), EINVAL), (dict(v=J + 2), EINVAL),
    (dict(v=I), EINVAL), (dict(k=A), EINVAL), (dict(v=C), EINVAL), (dict(k=H), EINVAL)])
def test_read_refuses(L, kw, status):
    assert read(L, **kw) == status


def test_nothing_to_read_is_ok_without_a_device(L):
    assert read(L, N=0, T=0, slots=0, k=0, v=0) == OK


def resize(L, fn="resize", refs=A, n_pages=64, table=B, lens=C, n_slots=8, max_pages=16, ps=16, slots=D_,
           new=E, n=4, layers=2, Hkv=2, Dh=64, block=16, k=F, v=G, kc=I, vc=J, ws=H, wsb=0):
    need = L.shortconv_pages_workspace_bytes(max(n_pages, 1), max(n, 0))
    return getattr(L, f"shortconv_pages_{fn}_8bit")(
        refs, n_pages, table, lens, n_slots, max_pages, ps, slots, new, n, layers, Hkv, Dh, block, k, v,
        kc, vc, ws, need + wsb, None)


@pytest.mark.parametrize("fn", ["resize", "fork"])
@pytest.mark.parametrize("kw,status", [
    (dict(block=32), EUNSUPPORTED), (dict(Dh=8), EUNSUPPORTED), (dict(Hkv=0), EINVAL), (dict(kc=0), EINVAL),
    (dict(vc=J + 1), EINVAL), (dict(kc=F + 64), EINVAL), (dict(vc=I), EINVAL), (dict(new=I), EINVAL),
    (dict(layers=-1), EINVAL), (dict(wsb=-1), EINVAL), (dict(ps=512), EUNSUPPORTED), (dict(n=9), EINVAL)])
def test_resize_and_fork_refuse(L, fn, kw, status):
    assert resize(L, fn=fn, **kw) == status


def test_nothing_listed_is_ok_without_a_device(L):
    assert resize(L, n=0, slots=0, new=0) == OK


def test_compact_refuses(L):
    def call(block=16, kc=I, vc=J, used=E):
        return L.shortconv_pages_compact_8bit(A, 64, B, C, 8, 16, 16, 1, 2, 64, block, F, G, kc, vc, used,
                                              H, L.shortconv_pages_workspace_bytes(64, 0), None)
    assert call(block=5) == EUNSUPPORTED
    assert call(kc=0) == EINVAL
    assert call(vc=I) == EINVAL
    assert call(used=I) == EINVAL


def attention(L, Hq=4, Hkv=2, Dh=64, block=16, q=A, qs=256, N=3, D=2, kp=B, vp=C, kc=D_, vc=E, n_pages=64,
              ps=32, table=F, lens=G, n_slots=8, max_pages=16, slots=H, shared=2, scale=0.125, out=I, ws=J,
              wsb=0):
    need = L.shortconv_prefix_attention_8bit_workspace_bytes(Hq, Hkv, Dh, N, D, shared, ps)
    return L.shortconv_prefix_attention_8bit(Hq, Hkv, Dh, block, q, qs, N, D, kp, vp, kc, vc, n_pages, ps,
                                             table, lens, n_slots, max_pages, slots, shared, scale, out,
                                             ws, need + wsb, None)


@pytest.mark.parametrize("kw,status", SHAPES + [
    (dict(Hq=5), EINVAL), (dict(Dh=32), EUNSUPPORTED), (dict(Hq=512), EINVAL), (dict(qs=255), EINVAL),
    (dict(qs=260), EUNSUPPORTED), (dict(N=-1), EINVAL), (dict(D=0), EINVAL), (dict(shared=17), EINVAL),
    (dict(scale=0.0), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(scale=1e31), EUNSUPPORTED),
    (dict(kc=0), EINVAL), (dict(vc=E + 2), EINVAL), (dict(out=D_), EINVAL), (dict(ws=E), EINVAL),
    (dict(out=A), EINVAL), (dict(q=0), EINVAL), (dict(kp=B + 8), EINVAL), (dict(wsb=-1), EINVAL)])
def test_attention_refuses(L, kw, status):
    assert attention(L, **kw) == status


def test_attention_workspace(L):
    f = L.shortconv_prefix_attention_8bit_workspace_bytes
    plain = L.shortconv_prefix_attention_workspace_bytes
    assert f(8, 2, 64, 3, 1, 0, 16) > 0
    unpacked = 2 * 5000 * 16 * 2 * 64 * 2
    prefix = plain(8, 2, 64, 3, 1, 5000) - plain(8, 2, 64, 3, 1, 0)
    assert f(8, 2, 64, 3, 1, 5000, 16) == f(8, 2, 64, 3, 1, 0, 16) + prefix + unpacked
    assert f(8, 2, 64, 3, 1, 4, 16) == f(8, 2, 64, 3, 1, 0, 16)  # few: read with the rest
    last = 0  # more shared pages never need less
    for shared in (0, 1, 64, 512, 2048, 4096, 4097, 8192, 65536):
        assert last <= f(8, 2, 64, 3, 1, shared, 16)
        last = f(8, 2, 64, 3, 1, shared, 16)
    for bad in ((8, 3, 64, 3, 1, 0, 16), (8, 2, 96, 3, 1, 0, 16), (8, 2, 64, -1, 1, 0, 16),
                (8, 2, 64, 3, 0, 0, 16), (8, 2, 64, 3, 1, -1, 16), (8, 2, 64, 3, 1, 1, 4),
                (8, 2, 64, 3, 1, 1 << 30, 16)):
        assert f(*bad) == 0


def rope(L, dt=BF16, layout=0, inv=0, Hq=4, Hkv=2, Dh=64, R=64, q=A, qs=256, k=B, ks=128, T=6, f=C, amp=1.0,
         pos=D_, lens=0, n_slots=0, slots=0, D=0, qo=E, qos=256, ko=F, kos=128):
    return L.shortconv_rope(dt, layout, inv, Hq, Hkv, Dh, R, q or None, qs, k or None, ks, T, f or None, amp,
                            pos or None, lens or None, n_slots, slots or None, D, qo or None, qos,
                            ko or None, kos, None)


BY_SLOT = dict(pos=0, lens=G, n_slots=5, slots=H, D=2)


@pytest.mark.parametrize("kw,status", [
    (dict(dt=2), EUNSUPPORTED), (dict(layout=2), EINVAL), (dict(Hq=-1), EINVAL), (dict(Hq=0, Hkv=0), EINVAL),
    (dict(Dh=0), EINVAL), (dict(R=0), EINVAL), (dict(R=63), EINVAL), (dict(R=66), EINVAL),
    (dict(T=-1), EINVAL), (dict(T=1 << 31), EINVAL), (dict(Dh=1024, R=514, qs=4096, ks=4096, qos=4096,
                                                           kos=4096), EUNSUPPORTED),
    (dict(qs=255), EINVAL), (dict(kos=127), EINVAL), (dict(ks=1 << 37), EUNSUPPORTED),
    (dict(q=0), EINVAL), (dict(q=A + 1), EINVAL), (dict(dt=F32, q=A + 2), EINVAL), (dict(ko=0), EINVAL),
    (dict(f=0), EINVAL), (dict(f=C + 4), EINVAL), (dict(pos=D_ + 2), EINVAL), (dict(pos=0), EINVAL),
    (dict(BY_SLOT, D=0), EINVAL), (dict(BY_SLOT, D=4), EINVAL), (dict(BY_SLOT, n_slots=0), EINVAL),
    (dict(BY_SLOT, lens=0), EINVAL), (dict(BY_SLOT, slots=H + 2), EINVAL), (dict(qo=B), EINVAL),
    (dict(ko=A), EINVAL), (dict(ko=E), EINVAL), (dict(qo=C), EINVAL), (dict(ko=D_), EINVAL),
    (dict(BY_SLOT, qo=G), EINVAL), (dict(qo=A + 2), EINVAL), (dict(qo=A, qos=512), EINVAL),
    # rows that lie between another's rows, 16 bytes too near
    (dict(k=A + 512 - 16, qs=512, ks=512, qo=A, qos=512, ko=A + 512 - 16, kos=512), EINVAL)])
def test_rope_refuses(L, kw, status):
    assert rope(L, **kw) == status


def test_nothing_to_turn_is_ok_without_a_device(L):
    assert rope(L, T=0, q=0, k=0, pos=0, qo=0, ko=0) == OK


def test_binding_refuses_wrong_arguments():
    import torch
    f = torch.zeros(4, dtype=torch.float64)
    q = torch.zeros(2, 1, 8)
    with pytest.raises(ValueError):
        sc.rope(q, None, f, positions=None)
    with pytest.raises(ValueError):
        sc.rope(q, None, f, positions=torch.zeros(2, dtype=torch.int32), layout="other")
    with pytest.raises(ValueError):
        sc.rope(None, None, f, positions=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        sc.rope(q.half(), None, f, positions=torch.zeros(2, dtype=torch.int32))
    pages = torch.zeros(4, 16, 1, 64)
    with pytest.raises(TypeError):  # scales beside a cache that has none
        sc.pages_append(q, q, pages, pages, torch.zeros(1, 4), None, torch.zeros(1), 1, k_scales=pages,
                        v_scales=pages)
    k8, v8, ks, vs = sc.page_cache_8bit(4, 16, 1, 64, block=8, device="cpu")
    assert k8.dtype == torch.float8_e4m3fn and ks.shape == (4, 2, 1)
    with pytest.raises(ValueError):  # an 8-bit cache without its scales
        sc.pages_append(q, q, k8, v8, torch.zeros(1, 4), None, torch.zeros(1), 1)
    with pytest.raises(ValueError):
        sc.page_cache_8bit(4, 16, 1, 64, block=32, device="cpu")
