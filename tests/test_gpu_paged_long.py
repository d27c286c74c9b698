"""What the results are off by on average over long caches: values of one sign, small scores, so that each weight and
each sum is rounded to either side alike and a mean that is not zero shows sums that are cut off (the tensor cores
truncate what they add up)."""

import pytest
import torch

import block_quantized_matmul_lwq_b200 as lwq
from paged_util import TYPES, Problem
from test_gpu_paged import dev                                    # noqa: F401  (the module's device and workspace)

pytestmark = pytest.mark.gpu


def long_problem(dev, dtype, lens, H, Hkv, D, page, **kw):
    """Scores of about 0.3 N(0, 1); values between 0.5 and 1, times a factor of the column, so that results fall
    anywhere between the steps of a 16-bit type."""
    p = Problem(dev, dtype, lens, H, Hkv, D, page, poison=False, **kw)
    p.q *= 0.3
    g = torch.Generator(device=dev)
    g.manual_seed(kw.get("seed", 0) + 100)
    v = 0.5 + 0.5 * torch.rand(p.vc.shape, generator=g, device=dev)
    p.vc.copy_(v * (1 + torch.arange(D, device=dev) / D))
    return p


def relative_errors(p, out, rows, causal):
    """(out - exact) / exact in 64 bits for the rows (sequence, its i-th new token) given."""
    errs = []
    for b, i in rows:
        n = p.lens[b] - p.new[b] + i + 1 if causal else p.lens[b]
        j = torch.arange(p.prefix + n, device=p.dev)
        own = j >= p.prefix
        jj = torch.where(own, j - p.prefix, j)
        pages = torch.where(own, p.tables[b][torch.where(own, jj // p.page, 0)],
                            (p.prefix_pages if p.prefix else p.tables[b])[torch.where(own, 0, jj // p.page)]).long()
        k, v = (c[pages, :, jj % p.page].double().transpose(0, 1) for c in (p.kc, p.vc))
        q = p.q[p.cu[b] + i].double().view(p.Hkv, p.G, p.D)
        w = torch.softmax(torch.einsum("hgd,hnd->hgn", q, k) * p.scale, -1)
        ref = torch.einsum("hgn,hnd->hgd", w, v).reshape(p.H, p.D)
        errs.append((out[p.cu[b] + i].double() - ref) / ref)
    return torch.stack(errs)


def call(p, causal, out16):
    out = torch.full((p.T, p.H, p.D), float("nan"), dtype=TYPES[p.dtype] if out16 else torch.float32, device=p.dev)
    flags = lwq.LWQ_FLAG_OUT16 if out16 else 0
    if causal:
        lwq.lwq_attention_prefill(p.cache(), p.q, out, p.cu_d, p.T, p.H, p.scale, flags=flags)
    else:
        lwq.lwq_attention_paged(p.cache(), p.q, out, p.H, p.scale, flags=flags)
    torch.cuda.synchronize(p.dev)
    assert lwq.lwq_get_device_error() == lwq.LWQ_OK
    return out


# A 16-bit result: its own rounding, at most half a step, is uniform over the columns' values, so its mean over 128
# columns (rows of one cache differ little) is off by less than 6 / sqrt(12 * 128) half steps; sums are cut by at most
# 2^-23 of themselves per product of 16 keys, over the 16384 keys (bf16: 32768) after which they are taken out of the
# accumulator, and half of that on average, as they grow; and the sum of the weights, a rounded one of 1024 tiles, is
# off by 1024 / 2 * 2^-25 at most.
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("where", ["prefill", "prefix"])
def test_16_bit_results_over_131072_keys(dev, dtype, where):       # noqa: F811
    half = torch.finfo(TYPES[dtype]).eps / 2
    products = (16384 if dtype == "f16" else 32768) // 16
    mean_bound = 6 / (12 * 128) ** 0.5 * half + products / 2 * 2.0 ** -23 + 512 * 2.0 ** -25
    worst_bound = 2 * half + mean_bound      # one part per weight, and the result's rounding
    if where == "prefill":                   # 76 pairs of row tiles: each takes all the keys
        p = long_problem(dev, dtype, [131072], 16, 1, 128, 256, new=[1200], seed=1)
        e = relative_errors(p, call(p, True, True), [(0, 0), (0, 599), (0, 1199)], True)
    else:
        p = long_problem(dev, dtype, [3, 0] * 600, 16, 1, 128, 256, prefix=131072, seed=2)
        e = relative_errors(p, call(p, False, True), [(0, 0), (601, 0), (1199, 0)], False)
    print(f"mean {float(e.mean()):.2e} (bound {mean_bound:.2e}), worst {float(e.abs().max()):.2e}")
    assert abs(float(e.mean())) <= mean_bound
    assert float(e.abs().max()) <= worst_bound


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("where", ["prefill", "prefix"])
def test_16_bit_results_with_growing_scores(dev, dtype, where):    # noqa: F811
    """The maximum grows by 30 over 20000 keys, in steps and all along: what was taken out of the accumulator is
    rescaled each time.  Scores of up to 45 are off by 2^-19 of a weight each way."""
    half = torch.finfo(TYPES[dtype]).eps / 2
    if where == "prefill":
        p = long_problem(dev, dtype, [20000], 16, 1, 128, 256, new=[1200], seed=3)
        table, n = p.tables[0], 20000
    else:
        p = long_problem(dev, dtype, [3, 0] * 600, 16, 1, 128, 256, prefix=20000, seed=4)
        table, n = p.prefix_pages, 20000
    j = torch.arange(n, device=dev)
    ramp = 30.0 * j / n + 5.0 * (j // 6000)
    p.kc[table[j // 256].long(), 0, j % 256, 0] = (ramp / 16).to(TYPES[dtype])
    p.q[..., 0] = 16.0 / p.scale
    causal = where == "prefill"
    rows = [(0, 0), (0, 599), (0, 1199)] if causal else [(0, 0), (601, 0), (1199, 0)]
    e = relative_errors(p, call(p, causal, True), rows, causal)
    print(f"worst {float(e.abs().max()):.2e}")
    assert float(e.abs().max()) <= 2 * half + 2 * 2.0 ** -18 + 256 * 2.0 ** -23
