"""A workspace sized for the largest call of a server does for its smaller ones."""

import pytest

import block_quantized_matmul_lwq_b200 as lwq
from block_quantized_matmul_lwq_b200 import build as lwq_build


@pytest.fixture(scope="module", autouse=True)
def built():
    lwq_build.build()


def cache(B, Hkv=8, D=128, max_pages=128, prefix_len=0):
    return lwq.lwq_paged(lwq.LWQ_ACT_F16, None, None, None, None, B=B, Hkv=Hkv, D=D, page=64, max_pages=max_pages,
                         num_pages=1 << 12, prefix=None, prefix_len=prefix_len)


@pytest.mark.parametrize("Hkv,G", [(1, 1), (8, 4), (5, 16), (32, 1)])
def test_prefill_sizes_grow_with_the_call(Hkv, G):
    """Few tokens are cut into more parts than many: each size covers all that come before it."""
    most = 0
    for T in (1, 2, 7, 64, 65, 300, 1000, 2500, 5000, 40000):
        size = lwq.lwq_attention_prefill_workspace_size(cache(16, Hkv), T, Hkv * G)
        assert size >= most
        most = max(most, size)
    whole = lwq.lwq_attention_prefill_workspace_size(cache(16, Hkv, prefix_len=999), 2500, Hkv * G)
    for B, pages, prefix in ((1, 128, 999), (16, 1, 0), (3, 128, 0), (16, 7, 500)):
        assert lwq.lwq_attention_prefill_workspace_size(cache(B, Hkv, max_pages=pages, prefix_len=prefix), 2500,
                                                        Hkv * G) <= whole


@pytest.mark.parametrize("Hkv,G", [(1, 1), (8, 4), (5, 16), (32, 1)])
def test_decode_sizes_grow_with_the_batch(Hkv, G):
    most = 0
    for B in (1, 3, 16, 33, 64, 100, 129, 192, 200, 256, 257, 1000):
        size = lwq.lwq_attention_paged_workspace_size(cache(B, Hkv, prefix_len=16384), Hkv * G)
        assert size >= most
        most = max(most, size)
        for prefix in (0, 1, 500):
            assert lwq.lwq_attention_paged_workspace_size(cache(B, Hkv, prefix_len=prefix), Hkv * G) <= size
