"""Appending with frequencies up to the largest that a rotation takes, at the farthest positions."""

import pytest
import torch

import block_quantized_matmul_lwq_b200 as lwq
from paged_util import Problem
from test_gpu_paged import dev, run_append                        # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_append_large_frequencies(dev, layout):                    # noqa: F811
    p = Problem(dev, "f16", [40], 4, 2, 64, 16, new=[9], seed=12)
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2, 123456789, -987654321, 1, 0, 2 ** 30 + 7, -1]],
                       dtype=torch.int32)
    freq = [1000003.7, 1048576.0, -999999.1, 65537.25, 1234.5678, 7.5, 1.0, 0.001]
    rope = lwq.lwq_rope_init(16, inv_freq=freq, layout=lwq.LWQ_ROPE_HALF if layout == "half" else lwq.LWQ_ROPE_PAIRS)
    run_append(p, "f32", rope, pos.to(dev), rope_args=dict(rot=16, layout=layout, inv_freq=freq))
