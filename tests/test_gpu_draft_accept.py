"""Draft verification on the GPU against the definition in whole numbers: equal, not near."""
import numpy as np
import pytest
import torch

import lfm2_gated_short_gb300 as sc
from oracle import serving

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(N, D, V, dtype, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((N, D + 1, V), generator=g) * spread
    target = torch.softmax(z, -1).to(DT[dtype])
    zq = z[:, :D] + torch.randn((N, D, V), generator=g)
    draft = torch.softmax(zq, -1).to(DT[dtype])
    tokens = (torch.multinomial(draft.float().reshape(N * D, V), 1, generator=g).view(N, D)
              if D else torch.zeros((N, 0))).to(torch.int32)
    return target, draft, tokens, torch.rand((N, D + 1), generator=g)


def check(target, draft, tokens, u, n=None, err=0, rows=None):
    """rows: device tensors to use in place of target and draft (strided views)."""
    f64 = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    ref = serving.draft_accept(f64(target), f64(draft), tokens.numpy(), u.numpy(),
                               None if n is None else n.numpy())
    assert ref[0] == err
    t, d = rows or (target.cuda(), None if draft is None else draft.cuda())
    for _ in range(2):
        a, out = sc.draft_accept(t, d, tokens.cuda(), u.cuda(),
                                 n_drafts=None if n is None else n.cuda())
        assert sc.get_error() == err
        assert np.array_equal(a.cpu().numpy(), ref[1])
        assert np.array_equal(out.cpu().numpy(), ref[2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D,V", [(1, 1, 1), (1, 1, 2), (3, 2, 31), (2, 3, 33), (5, 8, 1000),
                                   (2, 40, 257), (1, 4, 32000), (3, 2, 50021), (2, 1, 140001)])
def test_equals_the_definition(dtype, N, D, V):
    check(*inputs(N, D, V, dtype, seed=N + D + V))


@pytest.mark.parametrize("V", [7, 4099])
def test_certain_drafts(V):
    target, _, tokens, u = inputs(16, 4, V, "f32", seed=V, spread=1.0)
    tokens[:, 0] = target[:, 0].argmax(-1).to(torch.int32)
    check(target, None, tokens, u)


def test_no_drafts_samples_one_token():
    target, _, tokens, u = inputs(9, 0, 517, "f32", seed=4)
    check(target, None, tokens, u)


def test_ragged_counts():
    target, draft, tokens, u = inputs(20, 5, 300, "bf16", seed=5)
    n = torch.arange(20, dtype=torch.int32) % 6
    check(target, draft, tokens, u, n)


@pytest.mark.parametrize("r", [0.0, 0.99999994, 0.5])
def test_edge_uniforms(r):
    target, draft, tokens, u = inputs(8, 3, 4500, "f32", seed=6)
    u[:, -1] = r
    u[:4, :-1] = 0.0
    u[4:, :-1] = 0.99999994
    check(target, draft, tokens, u)


def test_equal_distributions_and_an_empty_rest():
    target, _, tokens, u = inputs(6, 2, 900, "f32", seed=7)
    draft = target[:, :2].clone()
    u[:, 0] = 0.99999994
    check(target, draft, tokens, u)
    # nothing of p is left after q: the token is drawn from p itself
    draft = torch.ones_like(draft)
    check(target, draft, tokens, u)


def test_one_token_holds_everything():
    N, V = 4, 70000
    target = torch.zeros((N, 2, V))
    for i, t in enumerate((0, 1, V // 2, V - 1)):
        target[i, :, t] = 1.0
    tokens = torch.tensor([[0], [0], [V // 2], [5]], dtype=torch.int32)
    check(target, None, tokens, torch.full((N, 2), 0.7))


def test_ties_and_not_numbers():
    target = torch.full((4, 2, 64), 1 / 64)
    target[1, :, :32] = float("nan")
    target[2, :, 0] = float("inf")
    target[3, :, 3:9] = -1.0
    tokens = torch.tensor([[3], [4], [5], [6]], dtype=torch.int32)
    u = torch.tensor([[0.9, 0.5]] * 4)
    check(target, torch.full((4, 1, 64), 1 / 32), tokens, u)


def test_strided_rows():
    N, D, V = 3, 2, 1003
    target, draft, tokens, u = inputs(N, D, V, "bf16", seed=8)
    wide_t = torch.full((N, D + 1, V + 14), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_d = torch.full((N, D, V + 5), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_t[..., :V], wide_d[..., :V] = target.cuda(), draft.cuda()
    check(target, draft, tokens, u, rows=(wide_t[..., :V], wide_d[..., :V]))


def test_bad_data():
    target, draft, tokens, u = inputs(5, 3, 100, "f32", seed=9)
    tokens[1, 2], tokens[3, 0] = 100, -1
    check(target, draft, tokens, u, err=serving.BAD_TOKEN)
    tokens[1, 2], tokens[3, 0] = 0, 0
    n = torch.tensor([0, 4, 3, -1, 2], dtype=torch.int32)
    check(target, draft, tokens, u, n, err=serving.BAD_ACCEPTED)
    target[2] = 0.0
    check(target, None, tokens, u, err=serving.BAD_PROBS)


def test_offsets_past_32_bits():
    """Row 17001 of a [17010, 2, 131072] target lies past 2^32 elements."""
    N, V = 17010, 131072
    target = torch.zeros((N, 2, V), dtype=torch.bfloat16, device="cuda")
    pick = torch.randint(0, V, (N,), generator=torch.Generator().manual_seed(1))
    target[torch.arange(N), :, pick.cuda()] = 1.0
    tokens = pick.view(N, 1).to(torch.int32).cuda()
    a, out = sc.draft_accept(target, None, tokens, torch.full((N, 2), 0.5, device="cuda"))
    assert sc.get_error() == 0
    assert bool((a == 1).all()) and bool((out == tokens).all())
