"""Serving entry points refuse sizes whose products pass 64 bits, before any CUDA call: a product that
wrapped round would pass as a small one."""
import pytest

import lfm2_gated_short_gb300 as sc
from lfm2_gated_short_gb300 import build as sc_build

EINVAL, EUNSUPPORTED = 1, 2
BF16, F32 = 1, 0
A, B, C, D_, E, F, G, H = ((1 << 56) + i * (1 << 52) for i in range(8))  # far apart
MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def L():
    sc_build.build()
    return sc.lib()


def attention(L, N, D, Hq, Hkv, qs):
    return L.shortconv_prefix_attention(BF16, Hq, Hkv, 64, A, qs, N, D, B, C, 64, 16, D_, E, 8, 16, F, 0,
                                        0.125, G, H, 2 ** 62, None)


@pytest.mark.parametrize("N,D,Hq", [(MAX, MAX, 4), (MAX, MAX, 2 ** 16), (2 ** 30, 2 ** 30, 16),
                                    (2 ** 24, 2 ** 24, 2 ** 16)])
def test_attention_rows(L, N, D, Hq):
    assert attention(L, N, D, Hq, Hq, Hq * 64) == EUNSUPPORTED
    assert L.shortconv_prefix_attention_workspace_bytes(Hq, Hq, 64, N, D, 0) == 0


def test_attention_query_bytes(L):
    # 2^29 rows 2^35 elements of 2 bytes apart: 2^65 bytes
    assert attention(L, 2 ** 29 + 1, 1, 1, 1, 2 ** 35) == EINVAL


def test_append_bytes(L):
    # 2^28 rows 2^36 bytes apart
    for ks, vs in ((2 ** 36, 64), (64, 2 ** 36)):
        assert L.shortconv_pages_append(A, ks, B, vs, 2 ** 28 + 1, 1, 64, C, D_, 64, 16, E, F, 8, 16, G,
                                        None) == EINVAL


def test_pool_bytes(L):
    # 2^16 layers x 2^24 pages x 64 tokens x 2^18 bytes = 2^64
    need = L.shortconv_pages_workspace_bytes(2 ** 24, 4)
    for fn in (L.shortconv_pages_resize, L.shortconv_pages_fork):
        assert fn(A, 2 ** 24, B, C, 8, 16, 64, D_, E, 4, 2 ** 16, 2 ** 18, F, G, H, need, None) == EINVAL
    assert L.shortconv_pages_compact(A, 2 ** 24, B, C, 8, 16, 64, 2 ** 16, 2 ** 18, F, G, D_, H, need,
                                     None) == EINVAL


@pytest.mark.parametrize("N,D,ts,ds", [(2 ** 30 + 1, 0, 2 ** 32, 1000), (7 * 10 ** 8, 2, 1000, 2 ** 32)])
def test_acceptance_bytes(L, N, D, ts, ds):
    # more than 2^30 rows 2^32 elements of 4 bytes apart
    assert L.shortconv_draft_accept(F32, 1000, N, D, A, ts, B, ds, C, D_, E, F, G, None) == EINVAL


@pytest.mark.parametrize("ps,max_pages,ok", [(8, 2 ** 28 - 1, False), (8, 2 ** 28 - 31, False),
                                             (8, 2 ** 28 - 32, True), (32, 2 ** 26 - 1, False),
                                             (64, 2 ** 25 - 1, False), (256, 2 ** 23 - 1, True)])
def test_attention_tokens_of_a_sequence(L, ps, max_pages, ok):
    """Key numbers run up to a tile or two past a sequence's end, in 32 bits: at most 2^31 - 256 tokens."""
    need = L.shortconv_prefix_attention_workspace_bytes(4, 4, 64, 0, 1, 0)
    assert L.shortconv_prefix_attention(BF16, 4, 4, 64, A, 256, 0, 1, B, C, 64, ps, D_, E, 1, max_pages, F,
                                        0, 0.125, G, H, need, None) == (0 if ok else EUNSUPPORTED)
