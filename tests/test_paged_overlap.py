"""Results may not lie in the cache's own pages: refused before any launch."""

import pytest

import block_quantized_matmul_lwq_b200 as lwq
from block_quantized_matmul_lwq_b200 import build as lwq_build
from test_paged_abi import status

K, V, Q, OUT = 0x100000, 0x200000, 0x300000, 0x400000     # 16-byte aligned integers, never dereferenced
BYTES = 9 * 2 * 16 * 64 * 2                               # of a cache


@pytest.fixture(scope="module", autouse=True)
def built():
    lwq_build.build()


def cache():
    return lwq.lwq_paged(lwq.LWQ_ACT_F16, K, V, Q, Q, B=2, Hkv=2, D=64, page=16, max_pages=4, num_pages=9)


@pytest.mark.parametrize("base", [K, V])
@pytest.mark.parametrize("at", ["first", "inside", "last", "reaches in"])
def test_results_in_the_cache(base, at):
    row = 2 * 4 * 64                                      # elements of q_out and out
    for es in (2, 4):
        out = base + {"first": 0, "inside": 4096, "last": BYTES - 16, "reaches in": 16 - es * row}[at]
        flags = lwq.LWQ_FLAG_OUT16 if es == 2 else 0
        assert status(lwq.lwq_attention_paged, cache(), Q, out, 4, 0.1, flags=flags) == lwq.LWQ_ERR_INVALID_ARG
        assert status(lwq.lwq_attention_prefill, cache(), Q, out, None, 2, 4, 0.1, flags=flags) == lwq.LWQ_ERR_INVALID_ARG
        if es == 2:
            assert status(lwq.lwq_kv_append, cache(), None, lwq.LWQ_ACT_F16, Q, 512, Q, 512, Q, 512, out, 2,
                          4) == lwq.LWQ_ERR_INVALID_ARG
