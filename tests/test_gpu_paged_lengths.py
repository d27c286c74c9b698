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


def test_prefill_offsets_that_do_not_ascend(dev):                  # noqa: F811
    """Offsets that jump back give the sequences more pairs of row tiles than T tokens of B sequences can have.  Tokens
    are taken as those of the first sequence that holds them; what lies past the pairs that there are stays as it was,
    and no partial result past the workspace is read (7 pairs and one per sequence here, the last token's is the
    17th)."""
    p = Problem(dev, "f16", [1000], 4, 2, 64, 16, new=[999], seed=1)
    cu = torch.tensor([0, 999, 0, 999, 0, 1000], dtype=torch.int32, device=dev)
    cache = lwq.lwq_paged(lwq.LWQ_ACT_F16, p.kc, p.vc, p.tables.repeat(5, 1), p.lens_d.repeat(5), B=5, Hkv=2, D=64,
                          page=16, max_pages=p.max_pages, num_pages=p.num_pages)
    q = torch.cat([p.q, p.q[:1]])
    out = torch.full((1000, 4, 64), 5.0, device=dev)
    lwq.lwq_attention_prefill(cache, q, out, cu, 1000, 4, p.scale)
    assert lwq.lwq_last_launch_count() == 2     # the keys are split
    torch.cuda.synchronize(dev)
    assert (out[999] == 5.0).all()
    assert_attention(p, out[:999], True)
