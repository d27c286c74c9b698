"""A key far above all others (an attention sink), whose value is zero: the result is what the other keys' small
weights make of their values, so a weight lost below the 16-bit types' range is the whole result.

Scores are exact: the query is 1 in its first element, a key its score there and zeros else.  With N keys of score 0
and value 1 behind a sink of score g (natural log) and value 0, every element of the result is N / (N + e^g)."""

import math

import pytest
import torch

import block_quantized_matmul_lwq_b200 as lwq
from paged_util import TYPES, Problem
from test_gpu_paged import dev                                    # noqa: F401  (the module's device and workspace)

pytestmark = pytest.mark.gpu

GAPS = [0.0, 5.0, 10.0, 14.0, 15.0, 16.0, 17.0, 17.5]


def sink_problem(dev, dtype, gap, lens, H, Hkv, D, page, **kw):
    """The sink is the first key of the prefix, or of every sequence where there is none."""
    p = Problem(dev, dtype, lens, H, Hkv, D, page, **kw)
    p.q.zero_()
    p.q[..., 0] = 1.0
    p.scale = 1.0
    live = ~torch.isnan(p.kc)
    p.kc[live], p.vc[live] = 0.0, 1.0
    first = [int(p.prefix_h[0])] if p.prefix else [int(p.tables_h[b, 0]) for b in range(p.B) if p.lens[b] > 0]
    for page0 in first:
        p.kc[page0, :, 0, 0] = gap
        p.vc[page0, :, 0] = 0.0
    return p


def expected(p, gap, causal):
    rows = []
    for b in range(p.B):
        for i in range(p.new[b]):
            n = p.prefix + (p.lens[b] - p.new[b] + i + 1 if causal else p.lens[b]) - 1
            rows.append(n / (n + math.exp(gap)))
    return torch.tensor(rows, dtype=torch.float64, device=p.dev)[:, None, None]


def bound(dtype, gap, n, out16, lift):
    """Largest relative error.  fp16: weights are multiples of 2^-24 / 2^lift of the largest, rounded, so one of
    e^-gap is off by at most 2^(gap log2(e) - 25 - lift) of itself; bf16 has fp32's range.  Beside it the parts
    (2^-23 with two of fp16, 2^-25 with three of bf16, half a step with one), exponents of up to 2^5 rounded
    (2^-19 of the weight, in the sink's and the others'), sums of n weights, and at most 1024 keys' products (three
    parts each, half the sum on average, 2^-23 apiece) in an accumulator that truncates."""
    eps = torch.finfo(TYPES[dtype]).eps / 2
    e = 2.0 ** -18 + (64 + n / 128) * 2.0 ** -24 + 96 * 2.0 ** -23
    if dtype == "f16":
        e += 2.0 ** (gap * math.log2(math.e) - 25 - lift)
    return e + (2 * eps if out16 else 2.0 ** -23)


def check(p, gap, causal, out16, lift):
    out = torch.full((p.T, p.H, p.D), float("nan"), dtype=TYPES[p.dtype] if out16 else torch.float32, device=p.dev)
    flags = lwq.LWQ_FLAG_OUT16 if out16 else 0
    if causal:
        lwq.lwq_attention_prefill(p.cache(), p.q, out, p.cu_d, p.T, p.H, p.scale, flags=flags)
    else:
        lwq.lwq_attention_paged(p.cache(), p.q, out, p.H, p.scale, flags=flags)
    torch.cuda.synchronize(p.dev)
    assert lwq.lwq_get_device_error() == lwq.LWQ_OK
    ref = expected(p, gap, causal)
    # 16-bit results below their type's normal range are multiples of its smallest step
    step = torch.finfo(out.dtype).smallest_normal * torch.finfo(out.dtype).eps if out16 else 0.0
    alone = (ref == 0).expand(out.shape)                           # rows that see the sink only
    assert (out[alone] == 0).all()
    err = float((((out.double() - ref).abs() - step) / ref)[~alone].max())
    n = p.prefix + max(p.lens)
    assert err <= bound(p.dtype, gap, n, out16, lift), f"relative error {err:.3e}"


@pytest.mark.parametrize("out16", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("gap", GAPS + [20.0])
def test_decode(dev, gap, dtype, out16):                           # noqa: F811
    check(sink_problem(dev, dtype, gap, [300, 4097, 65], 8, 2, 64, 16, seed=1), gap, False, out16, 15)
    check(sink_problem(dev, dtype, gap, [20000], 16, 1, 128, 64, seed=2), gap, False, out16, 15)


@pytest.mark.parametrize("out16", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("gap", GAPS)
def test_prefill(dev, gap, dtype, out16):                          # noqa: F811
    """Whole and with the keys split."""
    check(sink_problem(dev, dtype, gap, [300, 700, 65], 8, 2, 64, 16, new=[300, 130, 3], seed=3), gap, True, out16, 13)
    check(sink_problem(dev, dtype, gap, [9000], 16, 1, 128, 64, new=[7], seed=4), gap, True, out16, 13)
    check(sink_problem(dev, dtype, gap, [2500], 40, 40, 64, 64, new=[600], seed=5), gap, True, out16, 13)


@pytest.mark.parametrize("out16", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("gap", GAPS)
def test_prefix(dev, gap, dtype, out16):                           # noqa: F811
    """The sink and most keys in the prefix, some of the sequences' own, some with none."""
    check(sink_problem(dev, dtype, gap, [0, 300, 65], 8, 2, 64, 16, prefix=701, seed=6), gap, False, out16, 13)
    check(sink_problem(dev, dtype, gap, [5] * 90, 8, 8, 128, 64, prefix=3001, seed=7), gap, False, out16, 13)


@pytest.mark.parametrize("gap", [10.0, 14.0, 17.0])
@pytest.mark.parametrize("count", [3, 9])
def test_several_sinks(dev, gap, count):                           # noqa: F811
    """The first keys alike: few leave some of the tile's quarters without one, nine do not (and begin at 2^10)."""
    p = sink_problem(dev, "f16", gap, [3000], 8, 8, 128, 16, new=[40], seed=9)
    p.kc[int(p.tables_h[0, 0]), :, :count, 0] = gap
    p.vc[int(p.tables_h[0, 0]), :, :count] = 0.0
    out = torch.full((p.T, p.H, p.D), float("nan"), device=dev)
    lwq.lwq_attention_prefill(p.cache(), p.q, out, p.cu_d, p.T, p.H, p.scale)
    torch.cuda.synchronize(dev)
    n = torch.arange(2960, 3000, dtype=torch.float64, device=dev)[:, None, None] + 1 - count
    ref = n / (n + count * math.exp(gap))
    err = float(((out.double() - ref).abs() / ref).max())
    assert err <= bound("f16", gap, 3000, False, 15 if count == 3 else 10), f"relative error {err:.3e}"


def test_scores_far_beyond_the_lift(dev):                          # noqa: F811
    """Scores of 2^24 and more, which leave no room for a shift of 15: the largest key alone counts (the next lies 2^15
    or more behind it), whichever comes first, and nothing overflows."""
    for size in (3.0e3, 1.2e4):
        p = Problem(dev, "f16", [400], 4, 2, 64, 16, new=[40], seed=8, poison=False)
        p.kc.zero_()
        p.q.zero_()
        p.q[..., 0] = size
        p.scale = 8192.0
        for j in range(400):
            p.kc[p.tables_h[0, j // 16], :, j % 16, 0] = float(j % 7) * 0.125 + 0.5
        out = torch.full((40, 4, 64), float("nan"), device=dev)
        lwq.lwq_attention_prefill(p.cache(), p.q, out, p.cu_d, 40, 4, p.scale)
        torch.cuda.synchronize(dev)
        _, v = p.rows(0, 400)
        for i in (0, 17, 39):
            best = [j for j in range(361 + i) if j % 7 == 6]
            want = v[:, best].mean(1).repeat_interleave(2, 0)
            assert float((out[i].double() - want).abs().max()) < 1e-5
