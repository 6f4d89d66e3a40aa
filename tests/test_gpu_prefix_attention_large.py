"""prefix_attention at sizes whose element counts pass 32 bits. Bound as in
test_gpu_prefix_attention.py."""
import numpy as np
import pytest
import torch

import lfm2_gated_short_gb300 as sc
from oracle import serving
from test_gpu_prefix_attention import EPS, i32

pytestmark = pytest.mark.gpu


def test_one_sequence_of_more_than_2_to_31_output_elements():
    """131136 drafts x 128 heads x 128: the rows of the last 64 tokens begin past 2^31 elements.
    100 cached tokens: only the last 100 drafts see keys (a tile and a bit of them, so that some
    items are joined from parts), the rows before are zeros."""
    D, Hq, Dh, n, ps = 2 ** 17 + 64, 128, 128, 100, 16
    g = torch.Generator().manual_seed(1)
    pages = -(-n // ps)
    k = torch.randn((pages, ps, 1, Dh), generator=g).bfloat16()
    v = torch.randn((pages, ps, 1, Dh), generator=g).bfloat16()
    q_end = torch.randn((n, Hq, Dh), generator=g).bfloat16()
    q = torch.zeros((D, Hq, Dh), dtype=torch.bfloat16, device="cuda")
    q[D - n:] = q_end.cuda()
    out = torch.full((D, Hq, Dh), 7.0, dtype=torch.bfloat16, device="cuda")
    table = np.arange(pages)[None]
    sc.prefix_attention(q, k.cuda(), v.cuda(), i32(table), i32([n]), i32([0]), D, out=out)
    assert sc.get_error() == 0
    for t in out[:D - n].split(2 ** 14):
        assert bool((t == 0).all())
    ref, mag = serving.attention(q_end.double().numpy(), k.double().numpy(), v.double().numpy(), table,
                                 [n], [0], n, Dh ** -0.5)
    got = out[D - n:].double().cpu().numpy()
    assert (np.abs(got - ref) <= 1.5 * EPS * mag + 1.01 * EPS * np.abs(ref) + 2.0 ** -40).all()
