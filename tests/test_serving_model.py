"""The serving operators' plain definitions against closed forms and invariants (CPU)."""
import numpy as np
import pytest

from oracle import serving


def check_invariants(c):
    counts = np.zeros(c.n_pages, np.int64)
    for s, n in enumerate(c.lens):
        used = c.table[s, :c.pages(n)]
        assert (used >= 0).all() and (c.table[s, c.pages(n):] == -1).all()
        np.add.at(counts, used, 1)
        if n % c.ps:
            assert c.refs[used[-1]] == 1, "a partly filled last page is shared"
    assert np.array_equal(counts, c.refs)


def content(c, s):
    t = np.arange(c.lens[s])
    return c.k[:, c.table[s][t // c.ps], t % c.ps], c.v[:, c.table[s][t // c.ps], t % c.ps]


@pytest.mark.parametrize("seed", range(4))
def test_random_histories_keep_every_sequence(seed):
    r = np.random.default_rng(seed)
    c = serving.Cache(n_slots=7, max_pages=6, n_pages=24, page_size=8, L=2, width=3, rng=r)
    for _ in range(60):
        op = r.integers(3)
        before = [content(c, s) for s in range(7)]
        lens = c.lens.copy()
        if op == 0:
            slots = r.permutation(7)[:r.integers(1, 4)]
            new = r.integers(0, 49, len(slots))
            if c.resize(slots, new) == 0:
                lens[slots] = np.minimum(lens[slots], new)
        elif op == 1:
            p = r.permutation(7)
            if c.fork(p[:2], p[2:4]) == 0:
                for s, d in zip(p[:2], p[2:4]):
                    before[d], lens[d] = before[s], lens[s]
        else:
            used = c.compact()
            assert (c.refs[:used] > 0).all() and (c.refs[used:] == 0).all()
        check_invariants(c)
        for s in range(7):
            for new, old in zip(content(c, s), before[s]):
                assert np.array_equal(new[:, :lens[s]], old[:, :lens[s]])


def test_a_call_without_enough_pages_changes_nothing():
    c = serving.Cache(3, 4, 5, 8)
    assert c.resize([0, 1], [16, 17]) == 0
    before = c.refs.copy(), c.table.copy(), c.lens.copy()
    assert c.resize([0, 2], [8, 17]) == serving.NO_PAGE
    assert all(np.array_equal(x, y) for x, y in zip(before, (c.refs, c.table, c.lens)))


def test_attention_of_equal_keys_is_the_mean_of_the_values():
    r = np.random.default_rng(3)
    k = np.zeros((4, 8, 1, 64))
    v = r.standard_normal((4, 8, 1, 64))
    table, lens = np.array([[2, 0, 1]]), np.array([19])
    out, mag = serving.attention(r.standard_normal((2, 2, 64)), k, v, table, lens, [0], 2, 0.1)
    flat = np.concatenate([v[2], v[0], v[1]])[:, 0]
    for j, n in ((0, 18), (1, 19)):
        np.testing.assert_allclose(out[j], np.broadcast_to(flat[:n].mean(0), (2, 64)))
        np.testing.assert_allclose(mag[j], np.broadcast_to(np.abs(flat[:n]).mean(0), (2, 64)))


def test_attention_of_a_dominant_key_is_its_value_and_rows_without_keys_are_zero():
    k = np.zeros((1, 8, 1, 64))
    v = np.arange(8 * 64, dtype=float).reshape(1, 8, 1, 64)
    k[0, 3] = 1.0
    q = np.full((2, 1, 64), 50.0)
    out, _ = serving.attention(q, k, v, np.array([[0]]), np.array([6]), [0], 2, 1.0)
    np.testing.assert_allclose(out, np.broadcast_to(v[0, 3], (2, 1, 64)))
    out, _ = serving.attention(q, k, v, np.array([[0]]), np.array([1]), [0], 2, 1.0)
    assert (out[0] == 0).all() and (out[1] == v[0, 0]).all()


def test_accepted_drafts_and_the_next_token_follow_the_target():
    """Speculative sampling's output distribution is the target's: with every draft
    token and a fine grid of uniforms, the first output token has probabilities p."""
    p = np.array([0.5, 0.25, 0.125, 0.125])
    q = np.array([0.125, 0.5, 0.25, 0.125])
    target = np.stack([p, p])[None]
    counts = np.zeros(4)
    n = 64
    for x in range(4):
        for ua in range(n):
            for ub in range(n):
                u = np.array([[(ua + 0.5) / n, (ub + 0.5) / n]])
                err, a, out = serving.draft_accept(target, q[None, None], np.array([[x]]), u)
                assert err == 0 and a[0] in (0, 1)
                counts[out[0, 0]] += q[x] / n ** 2
    np.testing.assert_allclose(counts, p, atol=1.0 / n)


def test_certain_drafts_leave_the_target_without_the_draft():
    p = np.array([0.5, 0.0, 0.5])
    u = np.array([[0.75, 0.999]])
    err, a, out = serving.draft_accept(np.stack([p, p])[None], None, np.array([[0]]), u)
    assert (err, a[0], list(out[0])) == (0, 0, [2, -1])
    u[0, 0] = 0.25
    err, a, out = serving.draft_accept(np.stack([p, p])[None], None, np.array([[0]]), u)
    assert (err, a[0], list(out[0])) == (0, 1, [0, 2])


def test_zero_and_bad_inputs():
    z = np.zeros((1, 2, 3))
    assert serving.draft_accept(z, None, np.array([[1]]), np.zeros((1, 2)))[0] == serving.BAD_PROBS
    assert serving.draft_accept(z, None, np.array([[3]]), np.zeros((1, 2)))[0] == serving.BAD_TOKEN
    bad = serving.draft_accept(z, None, np.array([[0]]), np.zeros((1, 2)), n_drafts=[2])
    assert bad[0] == serving.BAD_ACCEPTED and (bad[2] == -1).all()
