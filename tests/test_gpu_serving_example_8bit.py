"""The serving example with rotary positions and an 8-bit cache: it runs, and its cache holds what the
first attention layer's keys and values quantise to."""
import numpy as np
import pytest
import torch

import lfm2_gated_short_gb300 as sc
from cache8_util import codes_from, i32, same_codes
from oracle import cache8
from test_gpu_serving_example import ex  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rotary,bits", [(64, 8), (32, 16), (0, 8)])
def test_generate(ex, rotary, bits):  # noqa: F811
    model = ex.Decoder(seed=1, rotary=rotary, context_factor=4.0, cache_bits=bits)
    g = torch.Generator(device="cuda").manual_seed(3)
    prompt = torch.randint(0, model.V, (40,), generator=g, device="cuda", dtype=torch.int32)
    sequences, counts, s, slots = ex.generate(model, prompt, 5, 3, 6)
    assert 0 <= int(counts.min()) and int(counts.max()) <= 3
    for b, seq in enumerate(sequences):
        assert int(s["lens"][int(slots[b])]) == 40 + len(seq) - 1
    assert sc.get_error() == 0


def test_the_prompt_in_the_cache(ex):  # noqa: F811
    model = ex.Decoder(seed=2, rotary=32, context_factor=4.0, cache_bits=8)
    T, slot = 45, torch.zeros(1, dtype=torch.int32, device="cuda")
    prompt = torch.arange(T, dtype=torch.int32, device="cuda") * 7 % model.V
    s = model.state(1, 4, 5, 16)
    ex.resize(s, slot, torch.full((1,), T, dtype=torch.int32, device="cuda"))
    pools = [s[x][0].clone() for x in ("k_scales", "v_scales")]
    model.forward(s, slot, prompt[None])
    # The first attention layer's input, by the same calls.
    x = model.embed[prompt.long()]
    conv = model.conv[0]
    bcx = (ex._norm(x) @ conv["w_in"].t()).contiguous()
    _, y = sc.verify(bcx, conv["w"], slot, torch.zeros_like(s["conv"][0]), T)
    x = x + y @ conv["w_out"].t()
    qkv = ex._norm(x) @ model.attn[0]["wqkv"].t()
    q, k, v = qkv.unflatten(1, (-1, model.Dh)).split((model.Hq, model.Hkv, model.Hkv), 1)
    _, k = sc.rope(None, k, model.freqs, positions=i32(range(T)), amplitude=model.amplitude)
    for name, new, scales in (("k", k, pools[0]), ("v", v, pools[1])):
        codes, want = np.zeros(s[name][0].shape, np.uint8), scales.cpu().numpy()
        assert cache8.append(codes, want, new.double().cpu().numpy(), s["table"].cpu().numpy(), [T], [0], T) == 0
        assert same_codes(codes_from(s[name][0]), codes)
        assert np.array_equal(s[name + "_scales"][0].cpu().numpy(), want)


def test_command_line(ex, monkeypatch, capsys):  # noqa: F811
    monkeypatch.setattr("sys.argv", ["x", "--branches", "3", "--steps", "2", "--prompt", "50", "--rotary", "64",
                                     "--cache-bits", "8"])
    ex.main()
    assert "drafts accepted" in capsys.readouterr().out
