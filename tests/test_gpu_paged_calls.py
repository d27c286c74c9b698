"""Calls of the paged cache that the documentation allows: a captured prefill replayed with other lengths and offsets,
keys alone with a rotation and the fewest threads, raw 16-bit storage."""

import pytest
import torch

import block_quantized_matmul_lwq_b200 as lwq
from paged_util import Problem, assert_attention, expected_append
from test_gpu_paged import dev                                    # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out16", [False, True])
@pytest.mark.parametrize("T", [40, 700])
def test_prefill_captured_and_replayed(dev, T, out16):             # noqa: F811
    """One graph for T rows of three sequences: whatever their lengths and offsets are when it is replayed; rows behind
    the last sequence stay.  T 40: the keys are split."""
    p = Problem(dev, "bf16", [1024] * 3, 8, 2, 64, 16, new=[T // 3] * 3, seed=1, poison=False)
    q = torch.randn((T, 8, 64), generator=torch.Generator().manual_seed(2)).bfloat16().to(dev)
    out = torch.empty((T, 8, 64), dtype=torch.bfloat16 if out16 else torch.float32, device=dev)
    cache, s = p.cache(), torch.cuda.Stream(dev)
    flags = lwq.LWQ_FLAG_OUT16 if out16 else 0

    def step():
        lwq.lwq_attention_prefill(cache, q, out, p.cu_d, T, 8, p.scale, flags=flags, stream=s)

    torch.cuda.synchronize(dev)
    step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for new, lens in (([T, 0, 0], [1000, 3, 0]), ([1, T - 9, 2], [1, 900, 1024]), ([0, 5, T // 2], [0, 5, T // 2])):
        p.new, p.lens, p.T = new, lens, sum(new)
        p.cu = [0, new[0], new[0] + new[1], sum(new)]
        p.lens_d.copy_(torch.tensor(lens, dtype=torch.int32))
        p.cu_d.copy_(torch.tensor(p.cu, dtype=torch.int32))
        p.q = q[:p.T]
        out.fill_(5.0)
        torch.cuda.synchronize(dev)
        graph.replay()
        torch.cuda.synchronize(dev)
        assert (out[p.T:] == 5.0).all()
        assert_attention(p, out[:p.T], True, out16)
    del graph


@pytest.mark.parametrize("D", [64, 128])
def test_append_keys_alone_with_a_rotation(dev, D):                # noqa: F811
    """One kv head and no queries: two warps, whose 64 threads turn up to 64 pairs."""
    p = Problem(dev, "f16", [30, 5], 1, 1, D, 16, new=[9, 5], seed=3)
    x = torch.randn((14, 3 * D), generator=torch.Generator().manual_seed(4)).to(dev)
    lwq.lwq_kv_append(p.cache(), lwq.lwq_rope_init(D), lwq.LWQ_ACT_F32, None, 0, x[:, D:], 3 * D, x[:, 2 * D:], 3 * D, None,
                      14, 1, cu_tokens=p.cu_d)
    torch.cuda.synchronize(dev)
    assert lwq.lwq_get_device_error() == lwq.LWQ_OK
    place = [n - m + i for n, m in zip(p.lens, p.new) for i in range(m)]
    seq = [b for b, m in enumerate(p.new) for _ in range(m)]
    _, k, v = expected_append(p, x, torch.tensor([place]), dict(rot=D, layout="half", base=10000.0))
    for t, (b, c) in enumerate(zip(seq, place)):
        at = int(p.tables_h[b, c // 16])
        # a rounding to fp16, and 2^-21 of |a| + |b| for the rotation in fp32
        bound = 2.0 ** -11 * 1.0001 * k[t].abs() + 2 * float(x.abs().max()) * 2.0 ** -21 + torch.finfo(torch.float16).tiny
        assert ((p.kc[at, :, c % 16].double() - k[t]).abs() <= bound).all()
        assert torch.equal(p.vc[at, :, c % 16], v[t].half())


def test_raw_storage(dev):                                         # noqa: F811
    """A cache, queries and results held as 16-bit integers: the bits of the type that the call names."""
    p = Problem(dev, "bf16", [100, 7], 4, 2, 64, 16, seed=5)
    out = torch.zeros((2, 4, 64), dtype=torch.int16, device=dev)
    raw = lwq.lwq_paged(lwq.LWQ_ACT_BF16, p.kc.view(torch.int16), p.vc.view(torch.int16), p.tables, p.lens_d, B=2, Hkv=2,
                        D=64, page=16, max_pages=p.max_pages, num_pages=p.num_pages)
    lwq.lwq_attention_paged(raw, p.q.view(torch.int16), out, 4, p.scale, flags=lwq.LWQ_FLAG_OUT16)
    torch.cuda.synchronize(dev)
    assert_attention(p, out.view(torch.bfloat16), False, True)


@pytest.mark.parametrize("scale", [0.0, 1e-33, -1e-33])
@pytest.mark.parametrize("where", ["prefix", "prefill"])
def test_small_scales_with_large_products(dev, where, scale):      # noqa: F811
    """Queries and keys of 1e15 in size: products near 1e31 times a scale of 0 or 1e-33."""
    p = Problem(dev, "bf16", [100, 7], 4, 2, 64, 16, new=[90, 7] if where == "prefill" else None,
                prefix=0 if where == "prefill" else 200, seed=6)
    p.q *= 1e15
    p.kc *= 1e15
    p.scale = scale
    out = torch.zeros((p.T, 4, 64), device=dev)
    if where == "prefill":
        lwq.lwq_attention_prefill(p.cache(), p.q, out, p.cu_d, p.T, 4, scale)
    else:
        lwq.lwq_attention_paged(p.cache(), p.q, out, 4, scale)
    torch.cuda.synchronize(dev)
    assert_attention(p, out, where == "prefill")
