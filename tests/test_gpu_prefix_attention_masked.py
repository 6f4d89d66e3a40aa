"""prefix_attention: what a row does not see inside its own sequence or the shared part.

Drafts that come after a row's token, and the shared part past a shorter sequence's end, may hold
anything, NaN and infinities in V included: a weight of zero would not silence them. Bound as in
test_gpu_prefix_attention.py.
"""
import numpy as np
import pytest
import torch

import lfm2_gated_short_gb300 as sc
from test_gpu_prefix_attention import EPS, build, call, check, reference

pytestmark = pytest.mark.gpu


def poison(c, i, pos, what, k=True, v=True, head=None):
    """Token `pos` of listed sequence i holds `what` (in one kv head, or all)."""
    ps = c["k"].shape[1]
    page = int(c["table"][c["slots"][i], pos // ps])
    h = slice(None) if head is None else head
    for t, on in ((c["k"], k), (c["v"], v)):
        if on:
            t[page, pos % ps, h] = what


def rows_of(c, got, i, js):
    G = c["q"].shape[1]
    return got.reshape(len(c["slots"]), c["D"], G, -1)[i, js]


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("D,Hkv,G,ps,shared", [(2, 2, 4, 16, 0), (3, 1, 5, 8, 0), (8, 2, 4, 16, 0),
                                               (8, 1, 3, 64, 2), (40, 2, 1, 16, 0), (70, 1, 2, 32, 1),
                                               (5, 2, 16, 16, 4)])
def test_a_later_draft_is_not_seen(Dh, D, Hkv, G, ps, shared, what):
    """Keys and values of draft j0 are not finite: tokens before it are as ever, j0 and later ones are
    not finite where the formula is not. Lengths put the drafts at, across and off a tile's end."""
    lens = [shared * ps + n for n in (D, D + 1, 64, 64 + D // 2, 127 + D, 100 + D)]
    j0 = D // 2
    c = build(lens, shared=shared, ps=ps, D=D, Hkv=Hkv, G=G, Dh=Dh, seed=D)
    lens = c["lens"][c["slots"]]
    for i, n in enumerate(lens):
        if n - D + j0 >= shared * ps:  # not in the shared part
            poison(c, i, n - D + j0, what, k=False)
    ref, mag = reference(c, Dh ** -0.5)
    clean = np.isfinite(ref)
    got = call(c).double().cpu().numpy()
    assert sc.get_error() == 0
    assert np.isfinite(got)[clean].all()
    over = np.abs(got - ref)[clean] - (1.5 * EPS * mag + 1.01 * EPS * np.abs(ref) + 2.0 ** -40)[clean]
    assert (over <= 0).all(), over.max()
    assert not np.isfinite(got)[~clean].any()
    shape = (len(lens), D, Hkv * G, Dh)
    assert clean.reshape(shape)[:, :j0].all() and not clean.reshape(shape)[:, j0:][lens >= D + shared * ps].any()


@pytest.mark.parametrize("Dh", [64, 128])
def test_one_column_of_a_later_draft(Dh):
    """A single NaN and a single infinity, in different columns and heads, reach their columns alone."""
    c = build([150, 77], D=4, Hkv=2, G=4, Dh=Dh, seed=3)
    s = c["slots"]
    at = [(int(c["table"][s[i], (c["lens"][s[i]] - 2) // 16]), int(c["lens"][s[i]] - 2) % 16) for i in (0, 1)]
    c["v"][at[0][0], at[0][1], 1, Dh - 3] = float("nan")
    c["v"][at[1][0], at[1][1], 0, 5] = float("inf")
    ref, mag = reference(c, Dh ** -0.5)
    got = call(c).double().cpu().numpy()
    assert sc.get_error() == 0
    clean = np.isfinite(ref)
    assert (~clean).sum() == 2 * 4 * 2  # tokens 2 and 3, the group's 4 heads, one column a sequence
    assert (np.isfinite(got) == clean).all()
    over = np.abs(got - ref)[clean] - (1.5 * EPS * mag + 1.01 * EPS * np.abs(ref) + 2.0 ** -40)[clean]
    assert (over <= 0).all(), over.max()


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("D,N", [(1, 5), (3, 5), (2, 90)])
def test_the_shared_part_past_a_shorter_sequence(Dh, D, N, what):
    """Some sequences end inside the shared part; a token behind their ends is not finite."""
    c = build([64] * N, shared=4, ps=16, D=D, Dh=Dh, seed=N)
    for i in range(N):
        c["lens"][c["slots"][i]] = (64, 0, 1, 33, 50)[i % 5]
    keep = [i for i in range(N) if c["lens"][c["slots"][i]] < 60]
    poison(c, 0, 60, what)
    ref, mag = reference(c, Dh ** -0.5)
    got = call(c).double().cpu().numpy()
    assert sc.get_error() == 0
    shape = (N, D, -1)
    ref, got, mag = (np.asarray(a).reshape(shape)[keep] for a in (ref, got, np.broadcast_to(mag, ref.shape)))
    assert np.isfinite(ref).all() and np.isfinite(got).all()
    assert (np.abs(got - ref) <= 1.5 * EPS * mag + 1.01 * EPS * np.abs(ref) + 2.0 ** -40).all()


@pytest.mark.parametrize("Dh", [64, 128])
def test_drafts_that_begin_inside_the_shared_part(Dh):
    """len - D below the shared tokens: some rows see all of the shared part, some do not."""
    check(build([130, 128, 131, 128 + 64, 140], shared=8, ps=16, D=9, G=3, Dh=Dh, seed=6))
    check(build([128, 129], shared=16, ps=8, D=4, G=8, Dh=Dh, seed=7))
