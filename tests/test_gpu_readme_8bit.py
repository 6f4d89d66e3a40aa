"""README's step with positions and an 8-bit cache, run as it stands there."""
import pytest
import torch

import lfm2_gated_short_gb300 as sc
from test_gpu_readme_serving import block

pytestmark = pytest.mark.gpu


def test_a_step_and_reading_back():
    N, D, Hq, Hkv, layers = 5, 40, 8, 2, 2
    g = torch.Generator(device="cuda").manual_seed(3)
    qkv = torch.randn((layers, N * D, Hq + 2 * Hkv, 64), generator=g, device="cuda").bfloat16()
    given = qkv.clone()
    names = dict(torch=torch, sc=sc, N=N, D=D, Hq=Hq, Hkv=Hkv, layers=layers, n_slots=8, qkv=qkv,
                 slots=torch.arange(1, N + 1, dtype=torch.int32, device="cuda"),
                 length=torch.full((N,), D, dtype=torch.int32, device="cuda"))
    exec(block("### Positions, and the cache in 8 bits"), names)
    assert sc.get_error() == 0
    assert names["out"].shape == (N * D, Hq, 64) and names["keys"].shape == (N * D, Hkv, 64)
    # e4m3 keeps 2^-4 of a value, and 2^-10 of a block's scale, which is below the block's largest / 224
    for got, new in ((names["keys"], qkv[0, :, Hq:Hq + Hkv]), (names["values"], given[0, :, Hq + Hkv:])):
        new = new.float()
        assert ((got.float() - new).abs() <= 2.0 ** -4 * new.abs() + new.abs().max() / 224 * 2.0 ** -10).all()
