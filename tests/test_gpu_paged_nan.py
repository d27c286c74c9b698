"""A query that is not a number, or infinite, gives a result that is not a number, in its row alone."""

import pytest
import torch

import block_quantized_matmul_lwq_b200 as lwq
from paged_util import Problem
from test_gpu_paged import dev                                    # noqa: F401
from test_gpu_paged_long import call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("out16", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("where", ["decode", "prefix", "prefill", "prefill split", "prefill long"])
def test_queries(dev, where, dtype, out16, bad):                   # noqa: F811
    if where == "decode":
        p = Problem(dev, dtype, [40, 5000, 3], 8, 2, 64, 16, seed=1)
    elif where == "prefix":
        p = Problem(dev, dtype, [40, 0, 3], 8, 2, 64, 16, prefix=700, seed=2)
    elif where == "prefill":
        p = Problem(dev, dtype, [300] * 20, 8, 8, 64, 16, new=[300] * 20, seed=3)
    elif where == "prefill split":
        p = Problem(dev, dtype, [5000], 8, 2, 64, 16, new=[5], seed=4)
    else:                       # past where sums are taken out of the accumulator
        p = Problem(dev, dtype, [40000], 16, 16, 64, 64, new=[300], seed=5, poison=False)
    causal = where.startswith("prefill")
    good = call(p, causal, out16)
    assert torch.isfinite(good).all()
    # (rows that see several keys: an infinite query whose every score is -inf is a row that sees nothing)
    later = 250 if where == "prefill" else 0
    hit = [(p.T // 4 + later, 0), (p.T - 1, 7), (p.T // 2 + later, 3)]
    for t, h in hit:
        p.q[t, h, 5] = bad
    out = call(p, causal, out16)
    mask = torch.zeros((p.T, p.H), dtype=torch.bool, device=dev)
    for t, h in hit:
        mask[t, h] = True
        assert torch.isnan(out[t, h]).all()
    # (the row tiles rescale a warp's rows together, by 1 where a row needs none)
    assert torch.equal(out[~mask], good[~mask])
    assert lwq.lwq_get_device_error() == lwq.LWQ_OK
