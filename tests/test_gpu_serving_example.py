"""The serving example: its speculative steps leave the same state as one token at a time."""
import importlib.util
import os

import pytest
import torch

import lfm2_gated_short_gb300 as sc

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "speculative_serving.py")


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("speculative_serving", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def cached(s, layer, slot):
    n, ps = int(s["lens"][slot]), s["k"].shape[2]
    t = torch.arange(n, device="cuda")
    page = s["table"][slot].long()[t // ps]
    return s["k"][layer][page, t % ps], s["v"][layer][page, t % ps]


@pytest.mark.parametrize("prompt_len,drafts", [(40, 3), (33, 1), (5, 4)])
def test_speculative_steps_leave_the_state_of_single_steps(ex, prompt_len, drafts):
    model = ex.Decoder(seed=prompt_len)
    g = torch.Generator(device="cuda").manual_seed(3)
    prompt = torch.randint(0, model.V, (prompt_len,), generator=g, device="cuda", dtype=torch.int32)
    sequences, counts, s, slots = ex.generate(model, prompt, 5, drafts, 6)
    assert 0 <= int(counts.min()) and int(counts.max()) <= drafts and int(counts.max()) > 0
    n_used = int(sc.pages_compact(s["refs"], s["table"], s["lens"], s["k"], s["v"]))
    assert int((s["refs"] > 0).sum()) == n_used

    i32 = dict(dtype=torch.int32, device="cuda")
    for b, seq in enumerate(sequences):
        # Every token but the last one drawn went through the layers: replay them one by one.
        tokens = prompt.tolist() + seq[:-1]
        assert int(s["lens"][int(slots[b])]) == len(tokens)
        if b % 2:
            continue
        r = model.state(1, 40, 40, 16)
        one = torch.zeros(1, **i32)
        for n, token in enumerate(tokens, 1):
            ex.resize(r, one, torch.full((1,), n, **i32))
            _, tapes = model.forward(r, one, torch.full((1, 1), token, **i32))
            ex.advance(r, one, tapes, torch.ones(1, **i32), torch.full((1,), n, **i32))
        slot = int(slots[b])
        # Layer 0's keys come before any attention: the same but for the order of a matrix
        # product's sums. Later layers also see attention outputs of other splits.
        for layer in range(2):
            for got, ref in zip(cached(s, layer, slot), cached(r, layer, 0)):
                assert (got.float() - ref.float()).abs().max() < 0.15
                assert (got.float() - ref.float()).abs().mean() < 0.01
        assert (s["conv"][:, slot].float() - r["conv"][:, 0].float()).abs().max() < 0.3
    assert sc.get_error() == 0


def test_command_line(ex, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["x", "--branches", "3", "--steps", "2", "--prompt", "50"])
    ex.main()
    assert "drafts accepted" in capsys.readouterr().out
