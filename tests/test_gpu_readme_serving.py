"""README's serving loop, run as it stands there: a step keeps its newest token and the accepted drafts."""
import os

import pytest
import torch

import lfm2_gated_short_gb300 as sc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


def block(heading):
    text = open(os.path.join(ROOT, "README.md"), encoding="utf-8").read()
    return text.split(heading, 1)[1].split("```python\n", 1)[1].split("```", 1)[0]


def test_a_step_keeps_the_newest_token_and_the_accepted_drafts():
    N, D, V, T, Hq = 5, 3, 700, 200, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    i32 = dict(dtype=torch.int32, device="cuda")

    def bf16(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()
    target = torch.softmax(torch.randn((N, D + 1, V), generator=g, device="cuda") * 3, -1)
    names = dict(
        torch=torch, sc=sc, n_slots=8, layers=2, N=N, D=D, shared=T // 16,
        prompt_slot=torch.zeros(1, **i32), prompt_len=torch.full((1,), T, **i32),
        slots=torch.arange(1, N + 1, **i32), length=torch.full((N,), T, **i32),
        k_new=bf16(N * (D + 1), 8, 64), v_new=bf16(N * (D + 1), 8, 64), q=bf16(N * (D + 1), Hq, 64),
        target_probs=target, draft_probs=target[:, :D].contiguous(),
        drafts=target[:, :D].argmax(-1).to(torch.int32),
        uniforms=torch.rand((N, D + 1), generator=g, device="cuda"))
    names["uniforms"][:2] = 0.9999  # equal distributions: all accepted but where u q = p rounds
    exec(block("### Speculative serving"), names)
    assert sc.get_error() == 0
    kept = names["accepted"] + 1  # of the step's D + 1 tokens
    assert torch.equal(names["lens"][1:N + 1], T + kept)
    assert names["out"].shape == (N * (D + 1), Hq, 64)
    assert names["tokens"].shape == (N, D + 1)
