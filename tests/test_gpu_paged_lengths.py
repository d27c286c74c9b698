"""Prefill with lengths beyond what the page table holds: as with the largest length that it does."""

import pytest
import torch

import block_quantized_matmul_lwq_b200 as lwq
from paged_util import Problem, assert_attention
from test_gpu_paged import dev                                    # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,length", [(3, 64), (64, 64), (5, 4096), (200, 640)])
@pytest.mark.parametrize("prefix", [0, 33])
@pytest.mark.parametrize("over", [1, 5, 1000, 2 ** 31 - 1])
def test_prefill_length_beyond_the_table(dev, over, prefix, new, length):   # noqa: F811
    """Whole and split keys; a second sequence whose length fits."""
    p = Problem(dev, "f16", [length, 40], 4, 2, 64, 16, new=[new, 7], prefix=prefix, seed=new,
                max_pages=length // 16)
    p.lens_d[0] = min(length + over, 2 ** 31 - 1)
    out = torch.full((p.T, 4, 64), float("nan"), device=dev)
    lwq.lwq_attention_prefill(p.cache(), p.q, out, p.cu_d, p.T, 4, p.scale)
    torch.cuda.synchronize(dev)
    assert_attention(p, out, True)          # (p.lens still holds the length that the table does)
