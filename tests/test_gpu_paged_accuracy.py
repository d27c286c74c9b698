"""The precision that fp32 results are said to have, each part of it by a test that fails without it: the second and third
16-bit parts of a probability, the sums that the row tiles keep outside their accumulator, the products that the decode
pass adds in rounded fp32; and that a call repeated gives the same bits."""

import pytest
import torch

import block_quantized_matmul_lwq_b200 as lwq
from paged_util import TYPES, Problem
from test_gpu_paged import dev                                    # noqa: F401
from test_gpu_paged_long import call, long_problem, relative_errors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("where", ["decode", "prefix", "prefill"])
def test_two_keys(dev, dtype, D, where):                           # noqa: F811
    """Keys of score 0 and -a, values 0 and 1: e^-a / (1 + e^-a), for 200 x 4 values of a between 0.5 and 4 that are
    numbers of the type.  log2(e) rounded is off by 2^-25 of a score, the score in units of it by 2^-22 in the decode
    pass and 2^-21 behind a shift of up to 15 in the row tiles; an exponential by 2^-22, the parts by 2^-23, three more
    roundings of 2^-24.  (One part less leaves 2^-12 in fp16, 2^-17 in bf16.)"""
    B = 200
    if where == "prefix":
        p = Problem(dev, dtype, [0] * B, 8, 2, D, 16, prefix=2, seed=1)
    else:
        p = Problem(dev, dtype, [2] * B, 8, 2, D, 16, new=[2] * B if where == "prefill" else None, seed=1)
    live = ~torch.isnan(p.kc)
    p.kc[live], p.vc[live] = 0.0, 0.0
    first = p.prefix_h[:1] if where == "prefix" else p.tables_h[:, 0]
    p.kc[first.long(), :, 1, 0] = -1.0
    p.vc[first.long(), :, 1] = 1.0
    p.q.zero_()
    a = 0.5 + 3.5 * torch.rand((p.T, p.H), generator=torch.Generator().manual_seed(D), dtype=torch.float64)
    a = a.to(TYPES[dtype]).to(dev)
    p.q[..., 0] = a
    p.scale = 1.0
    out = call(p, where == "prefill", False).double()
    w = torch.exp(-a.double())
    ref = (w / (1 + w))[..., None]
    if where == "prefill":
        out, ref = out[1::2], ref[1::2]                            # (the first token sees the zero alone)
    err = float(((out - ref).abs() / ref).max())
    bound = 6 * 2.0 ** -25 + (2.0 ** -22 if where == "decode" else 2.0 ** -21) + 2.0 ** -22 + 2.0 ** -23 + 3 * 2.0 ** -24
    print(f"{err:.2e} (bound {bound:.2e})")
    assert err <= bound


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("where", ["decode", "prefix", "prefill", "prefill split"])
def test_mean_error_of_long_sums(dev, dtype, where):               # noqa: F811
    """Values of one sign over 40000 keys.  Roundings go either way and leave no mean; what is truncated does: the
    products of 16 keys, each off by at most 2^-23 of what they are added to.  The decode pass adds them to nothing
    (parts x 2^-23 of themselves); the row tiles to sums of up to 1024 keys, half as large on average."""
    parts = 2 if dtype == "f16" else 3
    if where == "decode":
        p = long_problem(dev, dtype, [40000] * 4, 16, 8, 128, 64, seed=1)
        rows, bound = [(0, 0), (3, 0)], parts * 2.0 ** -23 + 2.0 ** -22
    elif where == "prefix":
        p = long_problem(dev, dtype, [3, 0] * 150, 16, 4, 128, 64, prefix=40000, seed=2)
        rows, bound = [(0, 0), (299, 0)], 64 * parts / 2 * 2.0 ** -23 + 2.0 ** -21
    elif where == "prefill":
        p = long_problem(dev, dtype, [40000], 16, 4, 128, 64, new=[1300], seed=3)
        rows, bound = [(0, 0), (0, 1299)], 64 * parts / 2 * 2.0 ** -23 + 2.0 ** -21
    else:
        p = long_problem(dev, dtype, [40000], 8, 8, 64, 256, new=[64], seed=4)
        rows, bound = [(0, 0), (0, 63)], 64 * parts / 2 * 2.0 ** -23 + 2.0 ** -21
    e = relative_errors(p, call(p, where.startswith("prefill"), False), rows, where.startswith("prefill"))
    print(f"{where} mean {float(e.mean()):.2e} (bound {bound:.2e}), worst {float(e.abs().max()):.2e}")
    assert abs(float(e.mean())) <= bound


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("out16", [False, True])
def test_repeated_calls_give_the_same_bits(dev, dtype, out16):     # noqa: F811
    for p, causal in ((Problem(dev, dtype, [7, 0, 300] * 30, 16, 4, 128, 64, prefix=3000, seed=1, poison=False), False),
                      (Problem(dev, dtype, [3000, 900], 16, 4, 128, 64, new=[2000, 30], seed=2, poison=False), True),
                      (Problem(dev, dtype, [9000], 8, 2, 64, 16, new=[6], seed=3, poison=False), True)):
        first = call(p, causal, out16)
        for _ in range(3):
            assert torch.equal(first, call(p, causal, out16))
