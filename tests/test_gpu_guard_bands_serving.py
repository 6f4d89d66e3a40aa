"""Guard bands around every buffer the serving operators write, on ragged shapes.

As in test_gpu_guard_bands.py: bands of a fill pattern around each written buffer, exactly
sized workspaces, every call against the model. The bounds-checked tests shorten a
record, so that the kernels' own accesses to its end are refused.
"""
import numpy as np
import pytest
import torch

import lfm2_gated_short_gb300 as sc
from oracle import serving
from test_gpu_guard_bands import Banded
from test_gpu_pages import Pair, i32
from test_gpu_prefix_attention import EPS, build, reference

pytestmark = pytest.mark.gpu


def banded(t):
    return Banded(t.shape, t.dtype, t)


class BandedPair(Pair):
    """A cache whose tables, pools and workspaces lie between bands."""

    def __init__(self, *a, **kw):
        super().__init__(*a, **kw)
        self.bands = {}
        for name in ("k", "v", "refs", "table", "lens"):
            self.bands[name] = banded(getattr(self, name))
            setattr(self, name, self.bands[name].t)

    def call(self, f, n, *args):
        ws = Banded((sc.pages_workspace_bytes(self.refs.shape[0], n),), torch.uint8)
        out = f(self.refs, self.table, self.lens, *args, self.k, self.v, workspace=ws.t)
        ws.check("workspace")
        for name, b in self.bands.items():
            b.check(name)
        return out


@pytest.mark.parametrize("n_slots,max_pages,n_pages,ps,L", [(7, 5, 29, 8, 2), (40, 130, 531, 16, 1),
                                                             (3, 3, 7, 64, 3)])
def test_pages(n_slots, max_pages, n_pages, ps, L):
    r = np.random.default_rng(n_slots)
    p = BandedPair(n_slots, max_pages, n_pages, ps, L)
    for _ in range(6):
        slots = r.permutation(n_slots)[:max(1, n_slots // 2)]
        new = r.integers(0, min(max_pages, 2 * n_pages // n_slots) * ps + 1, len(slots))
        p.call(sc.pages_resize, len(slots), i32(slots), i32(new))
        p.check(p.m.resize(slots, new))
        q = r.permutation(n_slots)
        src, dst = np.repeat(q[:1], n_slots - 1), q[1:]
        p.call(sc.pages_fork, len(dst), i32(src), i32(dst))
        p.check(p.m.fork(src, dst))
        n_used = Banded((1,), torch.int32)
        ws = Banded((sc.pages_workspace_bytes(n_pages, 0),), torch.uint8)
        sc.pages_compact(p.refs, p.table, p.lens, p.k, p.v, n_used=n_used.t, workspace=ws.t)
        ws.check("workspace")
        n_used.check("n_used")
        assert int(n_used.t) == p.m.compact()
        p.check()


def test_append():
    p = BandedPair(5, 4, 12, 8, 1, Hkv=3, Dh=8)
    slots = [3, 1]
    p.call(sc.pages_resize, 2, i32(slots), i32([13, 32]))
    p.m.resize(slots, [13, 32])
    k = torch.randn((10, 3, 8), device="cuda").bfloat16()
    sc.pages_append(k, -k, p.k[0], p.v[0], p.table, p.lens, i32(slots), 5)
    flat = k.double().cpu().numpy().reshape(10, -1)
    p.m.append(0, flat, -flat, slots, 5)
    for name, b in p.bands.items():
        b.check(name)
    p.check()


def attention(c, trim=None):
    Hq, Hkv, Dh = c["q"].shape[1], c["k"].shape[2], c["q"].shape[2]
    out = Banded(c["q"].shape, torch.bfloat16)
    need = sc.prefix_attention_workspace_bytes(Hq, Hkv, Dh, len(c["slots"]), c["D"], c["shared"])
    ws = Banded((need,), torch.uint8)
    args = (c["q"].cuda(), c["k"].cuda(), c["v"].cuda(), i32(c["table"]), i32(c["lens"]),
            i32(c["slots"]), c["D"])
    torch.cuda.synchronize()
    if trim:
        sc.bounds_trim_next(*trim)
    sc.prefix_attention(*args, shared_pages=c["shared"], out=out.t, workspace=ws.t)
    ws.check("workspace")
    out.check("out")
    return out.t.double().cpu().numpy()


@pytest.mark.parametrize("shared,D,G,Hkv,Dh", [(0, 1, 1, 1, 64), (0, 3, 7, 2, 64), (0, 2, 5, 2, 128),
                                               (3, 1, 3, 2, 64), (9, 5, 7, 1, 128), (5, 8, 4, 2, 64),
                                               (4, 1, 128, 1, 64)])
def test_attention(shared, D, G, Hkv, Dh):
    c = build([shared * 16 + n for n in (9, 33, 200, 16, 70)], shared=shared, D=D, G=G, Hkv=Hkv,
              Dh=Dh, seed=G)
    ref, mag = reference(c, Dh ** -0.5)
    got = attention(c)
    assert sc.get_error() == 0
    over = np.abs(got - ref) - (1.5 * EPS * mag + 1.01 * EPS * np.abs(ref) + 2.0 ** -40)
    assert (over <= 0).all()


def accept(target, draft, tokens, u, trim=None):
    N, D = tokens.shape
    a, out = Banded((N,), torch.int32), Banded((N, D + 1), torch.int32)
    t, d = banded(target), banded(draft)
    args = (tokens.cuda(), u.cuda())
    torch.cuda.synchronize()
    if trim:
        sc.bounds_trim_next(*trim)
    sc.draft_accept(t.t, d.t, *args, accepted=a.t, out_tokens=out.t)
    for b, what in ((a, "accepted"), (out, "out_tokens"), (t, "target"), (d, "draft")):
        b.check(what)
    return a.t.cpu().numpy(), out.t.cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,D,V", [(1, 1, 3), (3, 2, 1001), (2, 5, 9007), (1, 2, 40003)])
def test_draft_accept(dtype, N, D, V):
    g = torch.Generator().manual_seed(V)
    target = torch.softmax(torch.randn((N, D + 1, V), generator=g) * 2, -1).to(dtype).cuda()
    draft = torch.softmax(torch.randn((N, D, V), generator=g) * 2, -1).to(dtype).cuda()
    tokens = torch.randint(0, V, (N, D), generator=g, dtype=torch.int32)
    u = torch.rand((N, D + 1), generator=g) * 0.5
    a, out = accept(target, draft, tokens, u)
    assert sc.get_error() == 0
    ref = serving.draft_accept(target.double().cpu().numpy(), draft.double().cpu().numpy(),
                               tokens.numpy(), u.numpy())
    assert np.array_equal(a, ref[1]) and np.array_equal(out, ref[2])


# ------------------------------------------------ the bounds-checked build refuses

def test_a_shortened_output_is_refused():
    if not sc.bounds_checked():
        return  # the standard build has no records
    c = build([40, 50], seed=5)
    got = attention(c, trim=(6, 256))  # the last two heads of the last row
    assert sc.get_error() == sc.DEV_OUT_OF_BOUNDS
    assert sc.bounds_take_first_bad() != 0
    ref, _ = reference(c, 0.125)
    assert np.abs(got[0] - ref[0]).max() < 0.02 and np.abs(got[1, :2] - ref[1, :2]).max() < 0.02


def test_a_shortened_table_is_refused():
    if not sc.bounds_checked():
        return  # the standard build has no records
    p = Pair(4, 4, 16, 8)
    p.resize([0, 3], [20, 32])
    torch.cuda.synchronize()
    sc.bounds_trim_next(1, 4)  # the table loses its last entry, which slot 3 uses
    sc.pages_resize(p.refs, p.table, p.lens, i32([3]), i32([8]), p.k, p.v)
    assert sc.get_error() & sc.DEV_OUT_OF_BOUNDS
    assert sc.bounds_take_first_bad() != 0


def test_a_shortened_row_of_probabilities_is_refused():
    if not sc.bounds_checked():
        return  # the standard build has no records
    V = 5000
    p = torch.full((1, 2, V), 1 / V, device="cuda")
    accept(p, p[:, :1].clone(), torch.zeros((1, 1), dtype=torch.int32), torch.full((1, 2), 0.5),
           trim=(0, 64))
    assert sc.get_error() & sc.DEV_OUT_OF_BOUNDS
    assert sc.bounds_take_first_bad() != 0
