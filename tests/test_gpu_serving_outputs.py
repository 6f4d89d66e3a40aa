"""Outputs that a serving call allocates while it runs on a stream given to it.

The block must not be one whose last use is still pending on the current stream: here a copy out of
a tensor of the output's size waits there behind a delay while the tensor is given back.
"""
import numpy as np
import pytest
import torch

import lfm2_gated_short_gb300 as sc
from test_gpu_draft_accept import inputs
from test_gpu_pages import i32
from test_gpu_prefix_attention import build

pytestmark = pytest.mark.gpu


def attention():
    c = build(np.full(64, 70), G=4, Hkv=4, seed=1)
    a = (c["q"].cuda(), c["k"].cuda(), c["v"].cuda(), i32(c["table"]), i32(c["lens"]), i32(c["slots"]), 1)
    return (lambda **kw: sc.prefix_attention(*a, **kw)), c["q"].shape, torch.bfloat16


def accept():
    a = [t.cuda() for t in inputs(700, 4, 50, "f32", seed=2)]
    return (lambda **kw: sc.draft_accept(*a, **kw)[1]), (700, 5), torch.int32


def compact():
    refs, table, lens = sc.page_cache(4, 8, 32)
    k = torch.zeros((1, 32, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    return (lambda **kw: sc.pages_compact(refs, table, lens, k, k.clone(), **kw)), (1,), torch.int32


@pytest.mark.parametrize("make", [attention, accept, compact])
def test_an_output_on_a_given_stream_is_that_streams(make):
    call, shape, dtype = make()
    want = call().clone()
    call(stream=torch.cuda.Stream())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(4):
        held = [torch.full(shape, 7, dtype=dtype, device="cuda") for _ in range(4)]
        copies = [torch.empty_like(t) for t in held]
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)  # about 10 ms on the current stream
        for t, c in zip(held, copies):
            c.copy_(t)
        del held, t
        out = call(stream=side)  # its inputs are ready; nothing orders it behind the copies
        torch.cuda.synchronize()
        assert sc.get_error() == 0
        assert torch.equal(out, want)
        assert all((c == 7).all() for c in copies)
        del out
