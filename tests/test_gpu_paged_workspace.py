"""One workspace, sized for the largest call of a server, serves its smaller ones."""

import pytest
import torch

import block_quantized_matmul_lwq_b200 as lwq
from paged_util import Problem, check_attention
from test_gpu_paged import WS_BYTES, _ARENA, dev                   # noqa: F401

pytestmark = pytest.mark.gpu


def test_sized_for_the_largest(dev):                               # noqa: F811
    sizes = [(1, [3]), (2, [1, 70]), (5, [1, 2, 200, 5, 9]), (5, [700, 300, 500, 400, 600])]
    big = Problem(dev, "f16", [2000] * 5, 8, 4, 64, 16, new=[2000] * 5, seed=1, poison=False)
    need = max(lwq.lwq_attention_prefill_workspace_size(big.cache(), big.T, 8), 256)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=dev)
    try:
        lwq.lwq_init(ws, need)
        for B, new in sizes:
            p = Problem(dev, "f16", [n + 900 for n in new], 8, 4, 64, 16, new=new, seed=B, max_pages=125)
            check_attention(p, causal=True)
        need = lwq.lwq_attention_paged_workspace_size(
            Problem(dev, "f16", [5] * 200, 8, 4, 64, 16, prefix=3000, seed=2, poison=False).cache(), 8)
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=dev)
        lwq.lwq_init(ws, need)
        for B in (1, 33, 70, 129, 200):
            check_attention(Problem(dev, "f16", [b % 6 for b in range(B)], 8, 4, 64, 16, prefix=3000, seed=B), causal=False)
    finally:
        torch.cuda.synchronize(dev)
        lwq.lwq_init(_ARENA[0], WS_BYTES)
