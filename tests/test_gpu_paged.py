"""The paged key/value cache on the GPU: append with rotation, decode, shared prefix, prefill, and a run of them
together, against plain 64-bit implementations (tests/paged_util.py)."""

import numpy as np
import pytest
import torch

import block_quantized_matmul_lwq_b200 as lwq
import oracle
from block_quantized_matmul_lwq_b200 import inputs
from gpu_util import to_device
from paged_util import (TYPES, Problem, append_inputs, assert_attention, check_attention, expected_append)

pytestmark = pytest.mark.gpu

WS_BYTES = 96 << 20
_ARENA = []


@pytest.fixture(scope="module")
def dev():
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    _ARENA.append(torch.full((WS_BYTES,), 0xFF, dtype=torch.uint8, device=d))   # its contents need no initial value
    lwq.lwq_init(_ARENA[0], WS_BYTES)
    lwq.lwq_get_device_error()
    yield d
    torch.cuda.synchronize(d)
    lwq.lwq_shutdown()
    _ARENA.clear()


# ---------------------------------------------------------------------- append
def run_append(p, src, rope, pos=None, x=None, rope_args=None, null_positions=False, pad=0):
    """Appends the problem's new tokens and checks q_out, the new rows and that nothing else moved."""
    if x is None:
        x, n = append_inputs(p, src)
    else:
        n = x.shape[1]
    T = p.T + pad
    q_out = torch.full((T, p.H, p.D), 77.0, dtype=TYPES[p.dtype], device=p.dev)
    k0, v0 = p.kc.clone(), p.vc.clone()
    if pad:
        x = torch.cat([x, torch.full((pad, n), float("nan"), dtype=x.dtype, device=p.dev)])
    xf = x.view(-1)
    lwq.lwq_kv_append(p.cache(), rope, lwq.ACT_DTYPES[src], xf, n, xf[p.H * p.D:], n,
                      xf[(p.H + p.Hkv) * p.D:], n, q_out, T, p.H, cu_tokens=p.cu_d,
                      positions=None if null_positions else pos, stream=None)
    torch.cuda.synchronize(p.dev)
    assert lwq.lwq_get_device_error() == lwq.LWQ_OK
    place = [n_ - m + i for n_, m in zip(p.lens, p.new) for i in range(m)]
    seq = [b for b, m in enumerate(p.new) for _ in range(m)]
    if null_positions:
        axes = 1 if rope is None else rope.axes
        pos = torch.tensor([[c + p.prefix for c in place]] * axes)
    q, k, v = expected_append(p, x[:p.T], pos, rope_args)
    live = torch.tensor([c >= 0 for c in place])
    # |cos|, |sin| to 2^-23 + 2^-24 (angle, function), two products and a sum in fp32 (3 roundings of 2^-24):
    # under 2^-21 of |a| + |b| <= 2 max|x|; then one rounding to the 16-bit type
    size = float(x[:p.T].double().abs().max())
    half = torch.finfo(TYPES[p.dtype]).eps / 2
    tiny = torch.finfo(TYPES[p.dtype]).tiny

    def close(got, want):
        err = (got.double() - want).abs()
        assert (err <= half * 1.0001 * want.abs() + 2 * size * 2.0 ** -21 + tiny).all(), float(err.max())

    close(q_out[:p.T][live], q[live.to(p.dev)])
    assert (q_out[:p.T][~live] == 77.0).all() and (q_out[p.T:] == 77.0).all()
    idx = [(int(p.tables_h[b, c // p.page]), c % p.page) for b, c in zip(seq, place) if c >= 0]
    pages = torch.tensor([i[0] for i in idx], device=p.dev, dtype=torch.long)
    offs = torch.tensor([i[1] for i in idx], device=p.dev, dtype=torch.long)
    close(p.kc[pages, :, offs], k[live.to(p.dev)])
    close(p.vc[pages, :, offs], v[live.to(p.dev)])
    k0[pages, :, offs] = p.kc[pages, :, offs]
    v0[pages, :, offs] = p.vc[pages, :, offs]
    assert torch.equal(p.kc.view(torch.int16), k0.view(torch.int16))     # nothing else was written
    assert torch.equal(p.vc.view(torch.int16), v0.view(torch.int16))
    return q_out


@pytest.mark.parametrize("src", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 32), (64, 16), (128, 112)])
@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_append(dev, src, dtype, D, rot, layout):
    p = Problem(dev, dtype, [5, 40, 17, 1], 6, 2, D, 16, new=[5, 3, 1, 1], seed=rot + D)
    pos = torch.randint(0, 4000, (1, p.T), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    rope = lwq.lwq_rope_init(rot, base=10000.0, layout=lwq.LWQ_ROPE_HALF if layout == "half" else lwq.LWQ_ROPE_PAIRS)
    run_append(p, src, rope, pos.to(dev), rope_args=dict(rot=rot, layout=layout, base=10000.0))


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_append_three_axes(dev, layout):
    """Time, height and width turn 8, 13 and 11 pairs; far, negative and extreme positions."""
    p = Problem(dev, "bf16", [33, 9], 4, 4, 64, 32, new=[33, 2], seed=5)
    g = torch.Generator().manual_seed(4)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (3, p.T), generator=g, dtype=torch.int64).to(torch.int32)
    pos[0, :4] = torch.tensor([-2 ** 31, 2 ** 31 - 1, 0, -1], dtype=torch.int32)
    rope = lwq.lwq_rope_init(64, base=5e5, layout=lwq.LWQ_ROPE_HALF if layout == "half" else lwq.LWQ_ROPE_PAIRS,
                             sections=[8, 13, 11])
    run_append(p, "f32", rope, pos.to(dev), rope_args=dict(rot=64, layout=layout, base=5e5, sections=[8, 13, 11]))


def test_append_default_positions_follow_the_prefix(dev):
    p = Problem(dev, "f16", [70, 3], 2, 1, 64, 16, new=[9, 3], prefix=50, seed=6)
    freq = [1.0 / (i + 1) for i in range(16)]
    run_append(p, "f16", lwq.lwq_rope_init(32, inv_freq=freq), rope_args=dict(rot=32, layout="half", inv_freq=freq),
               null_positions=True)


def test_append_without_rotation_is_a_copy(dev):
    """rope None: values of the cache's type come back bit for bit, infinities too."""
    p = Problem(dev, "bf16", [20, 1], 4, 2, 128, 16, new=[20, 1], seed=7)
    x, n = append_inputs(p, "bf16")
    x[0, :8] = float("inf")
    q_out = torch.zeros((p.T, p.H, p.D), dtype=torch.bfloat16, device=dev)
    lwq.lwq_kv_append(p.cache(), None, lwq.LWQ_ACT_BF16, x, n, x[:, p.H * p.D:], n, x[:, (p.H + p.Hkv) * p.D:], n,
                      q_out, p.T, p.H, cu_tokens=p.cu_d)
    torch.cuda.synchronize(dev)
    assert torch.equal(q_out.view(p.T, -1), x[:, :p.H * p.D])
    k, v = p.rows(0, 20)
    assert torch.equal(k.transpose(0, 1).reshape(20, -1), x[:20, p.H * p.D:(p.H + p.Hkv) * p.D].double())
    assert torch.equal(v.transpose(0, 1).reshape(20, -1), x[:20, (p.H + p.Hkv) * p.D:].double())


def test_append_padding_and_many_sequences(dev):
    """70 sequences (more than a warp), some with no new token, one shorter than its new tokens, rows behind the last."""
    g = np.random.default_rng(0)
    new = [int(n) for n in g.integers(0, 4, 70)]
    lens = [int(n + m) for n, m in zip(new, g.integers(0, 90, 70))]
    new[11], lens[11] = 3, 2
    p = Problem(dev, "f16", lens, 4, 2, 64, 16, new=new, seed=8)
    rope = lwq.lwq_rope_init(64)
    run_append(p, "f32", rope, rope_args=dict(rot=64, layout="half", base=10000.0), null_positions=True, pad=5)


def test_append_one_token_each_without_offsets(dev):
    """cu_tokens None: a captured decode batch with two padded rows (length 0)."""
    p = Problem(dev, "f16", [16, 0, 33, 0, 1], 8, 8, 64, 16, seed=9)
    x, n = append_inputs(p, "f32")
    q_out = torch.full((5, 8, 64), 77.0, dtype=torch.float16, device=dev)
    lwq.lwq_kv_append(p.cache(), None, lwq.LWQ_ACT_F32, x, n, x[:, 512:], n, x[:, 1024:], n, q_out, 5, 8)
    torch.cuda.synchronize(dev)
    assert lwq.lwq_get_device_error() == lwq.LWQ_OK
    for b, c in ((0, 15), (2, 32), (4, 0)):
        assert torch.equal(q_out[b].view(-1), x[b, :512].half())
        assert torch.equal(p.kc[p.tables_h[b, c // 16], :, c % 16].reshape(-1), x[b, 512:1024].half())
    assert (q_out[1] == 77.0).all() and (q_out[3] == 77.0).all()


def test_append_strides_and_keys_only(dev):
    """Separate k and v with row strides of their own, no q."""
    p = Problem(dev, "bf16", [12], 4, 4, 64, 16, new=[12], seed=10)
    k = torch.randn((12, 320), device=dev).to(torch.bfloat16)
    v = torch.randn((12, 264), device=dev).to(torch.bfloat16)
    lwq.lwq_kv_append(p.cache(), None, lwq.LWQ_ACT_BF16, None, 0, k, 320, v, 264, None, 12, 4, cu_tokens=p.cu_d)
    torch.cuda.synchronize(dev)
    kk, vv = p.rows(0, 12)
    assert torch.equal(kk.transpose(0, 1).reshape(12, -1), k[:, :256].double())
    assert torch.equal(vv.transpose(0, 1).reshape(12, -1), v[:, :256].double())


def test_append_bad_pages(dev):
    """A page outside the cache, and a token beyond the page table: dropped and reported; the others are stored."""
    p = Problem(dev, "f16", [16, 16, 40], 2, 2, 64, 16, seed=11, max_pages=3)
    p.tables[0, 0] = p.num_pages
    p.tables[1, 0] = -1
    p.lens_d[2] = 49
    x, n = append_inputs(p, "f16")
    k0, v0 = p.kc.clone(), p.vc.clone()
    q_out = torch.zeros((3, 2, 64), dtype=torch.float16, device=dev)
    lwq.lwq_kv_append(p.cache(), None, lwq.LWQ_ACT_F16, x, n, x[:, 128:], n, x[:, 256:], n, q_out, 3, 2)
    torch.cuda.synchronize(dev)
    assert lwq.lwq_get_device_error() == lwq.LWQ_ERR_BAD_PAGE
    assert lwq.lwq_get_device_error() == lwq.LWQ_OK
    assert torch.equal(p.kc.view(torch.int16), k0.view(torch.int16))
    assert torch.equal(p.vc.view(torch.int16), v0.view(torch.int16))
    assert torch.equal(q_out.view(3, -1), x[:, :128])


# ---------------------------------------------------------------------- decode
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(4, 4), (10, 2), (7, 1), (8, 1), (18, 2), (16, 1), (6, 2)])
@pytest.mark.parametrize("page", [16, 64])
def test_decode_heads(dev, dtype, D, H, Hkv, page):
    check_attention(Problem(dev, dtype, [1, 15, 16, 17, 150], H, Hkv, D, page, seed=H + D), causal=False)


@pytest.mark.parametrize("out16", [False, True])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_decode_lengths(dev, page, out16):
    """Empty, one, around tile and page edges, long; unused table entries name no page."""
    lens = [0, 1, 63, 64, 65, 127, 128, 129, 0, 255, 257, 1000, 2049, -3]
    check_attention(Problem(dev, "bf16", lens, 8, 2, 128, page, seed=page), causal=False, out16=out16)


def test_decode_every_sequence_empty(dev):
    check_attention(Problem(dev, "f16", [0, 0, 0], 4, 2, 64, 16, seed=1), causal=False)


@pytest.mark.parametrize("B,L", [(1, 20000), (3, 5001), (300, 70)])
def test_decode_division_of_the_keys(dev, B, L):
    """One long sequence over every CTA, a few, and more sequences than CTAs."""
    check_attention(Problem(dev, "f16", [L - (7 * b) % 50 for b in range(B)], 8, 2, 64, 32, seed=B), causal=False)


def test_decode_large_scores(dev):
    """Scores of several hundred either way: the running maximum keeps every exponential finite."""
    p = Problem(dev, "f16", [300, 77], 4, 2, 64, 16, seed=2)
    p.scale = 8.0
    check_attention(p, causal=False)
    p.scale = -8.0
    check_attention(p, causal=False)


def test_decode_scale_zero_is_the_mean(dev):
    p = Problem(dev, "bf16", [333, 1], 4, 2, 64, 16, seed=2)
    p.scale = 0.0
    check_attention(p, causal=False)


def test_decode_length_beyond_the_table(dev):
    """A length past max_pages * page counts as that."""
    p = Problem(dev, "f16", [64], 4, 2, 64, 16, seed=3)
    p.lens_d[0] = 1 << 20
    check_attention(p, causal=False)


def test_decode_bad_page_reads_as_zeros(dev):
    p = Problem(dev, "f16", [100, 100], 4, 2, 64, 16, seed=4)
    lwq.lwq_get_device_error()
    good = torch.zeros((2, 4, 64), device=dev)
    lwq.lwq_attention_paged(p.cache(), p.q, good, 4, p.scale)
    p.tables[0, 2] = 1 << 30
    out = torch.zeros_like(good)
    lwq.lwq_attention_paged(p.cache(), p.q, out, 4, p.scale)
    torch.cuda.synchronize(dev)
    assert lwq.lwq_get_device_error() == lwq.LWQ_ERR_BAD_PAGE
    assert torch.equal(out[1], good[1])
    page = int(p.tables_h[0, 2])
    p.kc[page], p.vc[page] = 0, 0
    p.tables[0, 2] = page
    check_attention(p, causal=False)
    ref, den, _ = p.expected(False)
    assert float(((out.double() - ref).abs() / den).max()) < 1e-4


def test_decode_offsets_past_32_bits(dev):
    """A cache of more than 2^32 elements whose last pages are the ones in use."""
    page, Hkv, D = 64, 8, 128
    pages = 2 ** 32 // (page * Hkv * D) + 70
    p = Problem(dev, "f16", [1500, 777], 16, Hkv, D, page, seed=5, new=[200, 3])
    big = [torch.empty((pages, Hkv, page, D), dtype=torch.float16, device=dev) for _ in range(2)]
    small_k, small_v, n = p.kc, p.vc, p.num_pages
    big[0][pages - n:], big[1][pages - n:] = small_k, small_v
    view = p.cache()
    high = torch.where(p.tables >= 0, p.tables + (pages - n), p.tables)
    view = lwq.lwq_paged(lwq.LWQ_ACT_F16, big[0], big[1], high, p.lens_d, B=2, Hkv=Hkv, D=D, page=page,
                         max_pages=p.max_pages, num_pages=pages)
    out = torch.zeros((p.T, 16, D), device=dev)
    lwq.lwq_attention_prefill(view, p.q, out, p.cu_d, p.T, 16, p.scale)
    torch.cuda.synchronize(dev)
    assert_attention(p, out, True)
    p.new, p.T, p.cu = [1, 1], 2, [0, 1, 2]
    p.q = p.q[:2].contiguous()
    out = torch.zeros((2, 16, D), device=dev)
    lwq.lwq_attention_paged(view, p.q, out, 16, p.scale)
    torch.cuda.synchronize(dev)
    assert_attention(p, out, False)
    x = torch.randn((2, 32 * D), device=dev)
    q_out = torch.zeros((2, 16, D), dtype=torch.float16, device=dev)
    lwq.lwq_kv_append(view, None, lwq.LWQ_ACT_F32, x, 32 * D, x[:, 16 * D:], 32 * D, x[:, 24 * D:], 32 * D, q_out, 2, 16)
    torch.cuda.synchronize(dev)
    for b, c in ((0, 1499), (1, 776)):
        assert torch.equal(big[0][int(high[b, c // page]), :, c % page].reshape(-1), x[b, 16 * D:24 * D].half())
    assert lwq.lwq_get_device_error() == lwq.LWQ_OK


def test_decode_is_deterministic(dev):
    p = Problem(dev, "bf16", [3000, 1, 700], 16, 4, 128, 16, seed=6, prefix=200)
    outs = [check_attention(p, causal=False) for _ in range(2)]
    assert torch.equal(outs[0], outs[1])


# ---------------------------------------------------------------------- prefix
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(4, 4), (6, 2), (16, 1)])
@pytest.mark.parametrize("prefix", [1, 16, 100, 129, 700])
def test_prefix(dev, dtype, D, H, Hkv, prefix):
    check_attention(Problem(dev, dtype, [0, 1, 33, 64, 5], H, Hkv, D, 16, prefix=prefix, seed=prefix), causal=False)


@pytest.mark.parametrize("B", [1, 9, 40, 130, 300])
def test_prefix_batches(dev, B):
    """Rows (sequences x heads of a kv head) from one tile to several."""
    lens = [(37 * b) % 41 for b in range(B)]
    check_attention(Problem(dev, "bf16", lens, 8, 2, 64, 32, prefix=300, seed=B), causal=False, out16=B == 40)


@pytest.mark.parametrize("page", [16, 64, 128, 256])
def test_prefix_long(dev, page):
    check_attention(Problem(dev, "f16", [10, 0, 300], 8, 2, 128, page, prefix=5003, seed=page), causal=False)


def test_prefix_alone(dev):
    """No sequence has a token of its own."""
    check_attention(Problem(dev, "f16", [0, 0], 4, 2, 64, 16, prefix=40, seed=1), causal=False)


def test_prefix_equals_the_same_pages_in_every_table(dev):
    """The prefix's pages at the head of each table instead: the same outputs to rounding."""
    p = Problem(dev, "bf16", [20, 64, 5], 8, 2, 128, 16, prefix=256, seed=2)
    shared = check_attention(p, causal=False)
    tables = torch.cat([p.prefix_pages.repeat(3, 1), p.tables], 1).contiguous()
    lens = p.lens_d + 256
    plain = lwq.lwq_paged(lwq.LWQ_ACT_BF16, p.kc, p.vc, tables, lens, B=3, Hkv=2, D=128, page=16,
                          max_pages=tables.shape[1], num_pages=p.num_pages)
    out = torch.zeros_like(shared)
    lwq.lwq_attention_paged(plain, p.q, out, 8, p.scale)
    torch.cuda.synchronize(dev)
    assert_attention(p, out, False)


def test_prefix_bad_page(dev):
    p = Problem(dev, "f16", [10, 3], 4, 2, 64, 16, prefix=100, seed=3)
    page = int(p.prefix_h[3])
    p.prefix_pages[3] = -5
    out = torch.zeros((2, 4, 64), device=dev)
    lwq.lwq_attention_paged(p.cache(), p.q, out, 4, p.scale)
    torch.cuda.synchronize(dev)
    assert lwq.lwq_get_device_error() == lwq.LWQ_ERR_BAD_PAGE
    p.kc[page], p.vc[page] = 0, 0
    assert_attention(p, out, False)


# --------------------------------------------------------------------- prefill
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (6, 2), (5, 1), (16, 1)])
def test_prefill_heads(dev, dtype, D, H, Hkv):
    check_attention(Problem(dev, dtype, [40, 9, 150, 1], H, Hkv, D, 16, new=[40, 3, 130, 1], seed=H), causal=True)


@pytest.mark.parametrize("out16", [False, True])
@pytest.mark.parametrize("prefix", [0, 77, 128])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_prefill_ragged(dev, page, prefix, out16):
    """Whole prompts, chunks of cached ones, drafts, a single token, no new token, more new tokens than the cache
    holds (their first rows see nothing), across tile edges."""
    new = [128, 1, 0, 129, 5, 260, 6, 64]
    lens = [128, 300, 40, 140, 511, 260, 4, 640]
    p = Problem(dev, "bf16", lens, 4, 2, 128, page, new=new, prefix=prefix, seed=page + prefix)
    check_attention(p, causal=True, out16=out16)


@pytest.mark.parametrize("new,length", [(1, 9000), (7, 9000), (64, 4100), (300, 2500)])
def test_prefill_few_tokens_long_cache(dev, new, length):
    """Drafted tokens and small chunks against long caches: the keys are split."""
    check_attention(Problem(dev, "f16", [length], 8, 2, 64, 64, new=[new], seed=new), causal=True)


def test_prefill_empty_rows_and_padding(dev):
    """lens 0 with new tokens (padding): zeros, even with a prefix; rows behind the last sequence stay."""
    p = Problem(dev, "f16", [0, 30], 4, 2, 64, 16, new=[4, 10], prefix=20, seed=1)
    out = torch.full((p.T + 9, 4, 64), 5.0, device=dev)
    q = torch.cat([p.q, torch.full((9, 4, 64), float("nan"), dtype=torch.float16, device=dev)])
    lwq.lwq_attention_prefill(p.cache(), q, out, p.cu_d, p.T + 9, 4, p.scale)
    torch.cuda.synchronize(dev)
    assert (out[p.T:] == 5.0).all()
    assert_attention(p, out[:p.T], True)


def test_prefill_large_scores(dev):
    p = Problem(dev, "bf16", [300], 4, 2, 128, 16, new=[300], seed=2)
    p.scale = 6.0
    check_attention(p, causal=True)
    p.scale = -6.0
    check_attention(p, causal=True)


def test_prefill_growing_scores(dev):
    """Scores that grow along the keys by far more than the accumulator is let run ahead: every tile rescales."""
    p = Problem(dev, "f16", [900], 2, 1, 64, 16, new=[200], seed=3, poison=False)
    ramp = torch.linspace(0, 30, 900)
    for j in range(900):
        p.kc[p.tables_h[0, j // 16], 0, j % 16] = ramp[j]
    p.q = torch.ones_like(p.q)
    check_attention(p, causal=True)
    for j in range(900):
        p.kc[p.tables_h[0, j // 16], 0, j % 16] = -ramp[j]
    check_attention(p, causal=True)


def test_prefill_without_offsets_is_decode(dev):
    p = Problem(dev, "f16", [30, 0, 500], 4, 2, 64, 16, prefix=33, seed=4)
    out = torch.zeros((3, 4, 64), device=dev)
    lwq.lwq_attention_prefill(p.cache(), p.q, out, None, 3, 4, p.scale)
    torch.cuda.synchronize(dev)
    assert_attention(p, out, True)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("ramp", [False, True])
def test_prefill_sums_kept_past_1024_keys(dev, dtype, ramp):
    """fp32 results over more keys than the accumulator sums at a time, whole (160 row tiles: no split) and split;
    with scores that grow, so that the kept sums have to be rescaled."""
    p = Problem(dev, dtype, [2400], 20, 20, 64, 64, new=[1800], seed=6)
    long = Problem(dev, dtype, [40000], 8, 8, 64, 256, new=[64], seed=7)
    if ramp:
        for q in (p, long):
            n = q.lens[0]
            j = torch.arange(n)
            up = (torch.arange(n) * (6.0 / n)).to(TYPES[dtype]).to(dev)
            q.kc[q.tables_h[0][j // q.page].long().to(dev), :, (j % q.page).to(dev), :4] = up[:, None, None]
            q.q[..., :4] = 4.0
    check_attention(p, causal=True)
    check_attention(long, causal=True)


@pytest.mark.parametrize("B", [90, 200])
def test_prefill_many_short_sequences(dev, B):
    new = [1 + (5 * b) % 7 for b in range(B)]
    lens = [n + (11 * b) % 60 for b, n in enumerate(new)]
    check_attention(Problem(dev, "f16", lens, 8, 4, 64, 16, new=new, seed=5), causal=True)


# ------------------------------------------------------------- streams, graphs
def test_captured_and_replayed(dev):
    """A decode step captured once: append, then attention with a prefix; replayed with new lengths and inputs."""
    p = Problem(dev, "f16", [60, 0, 47], 8, 2, 64, 16, prefix=40, seed=7, max_pages=6, spare=12)
    free = [i for i in range(p.num_pages) if i not in set(p.tables_h.flatten().tolist()) | set(p.prefix_h.tolist())]
    for b in range(3):       # the pages that later tokens will need
        for i in range(6):
            if p.tables_h[b, i] < 0:
                p.tables_h[b, i] = free.pop(0) if free else 0
    p.tables.copy_(p.tables_h)
    x, n = append_inputs(p, "f32")
    rope = lwq.lwq_rope_init(64)
    out = torch.zeros((3, 8, 64), device=dev)
    q16 = torch.zeros((3, 8, 64), dtype=torch.float16, device=dev)
    cache = p.cache()
    s = torch.cuda.Stream(dev)

    def step():
        lwq.lwq_kv_append(cache, rope, lwq.LWQ_ACT_F32, x, n, x[:, 512:], n, x[:, 640:], n, q16, 3, 8, stream=s)
        lwq.lwq_attention_paged(cache, q16, out, 8, p.scale, stream=s)

    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for it in range(3):
        p.lens = [61 + it, it, 48 + it]
        p.lens_d.copy_(torch.tensor(p.lens, dtype=torch.int32))
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(it)))
        torch.cuda.synchronize(dev)
        graph.replay()
        torch.cuda.synchronize(dev)
        p.q = q16.clone()
        assert_attention(p, out, False)
    del graph


def test_other_stream(dev):
    s = torch.cuda.Stream(dev)
    torch.cuda.synchronize(dev)
    check_attention(Problem(dev, "f16", [500, 3], 8, 2, 64, 16, prefix=150, seed=1), causal=False, stream=s)
    check_attention(Problem(dev, "f16", [500, 3], 8, 2, 64, 16, new=[200, 3], seed=1), causal=True, stream=s)


def test_workspace_is_checked(dev):
    p = Problem(dev, "f16", [5000], 8, 2, 64, 16, seed=1)
    need = lwq.lwq_attention_paged_workspace_size(p.cache(), 8)
    assert need > 0
    small = torch.zeros(64, dtype=torch.uint8, device=dev)
    out = torch.zeros((1, 8, 64), device=dev)
    try:
        lwq.lwq_init(small, 64)
        with pytest.raises(lwq.LwqError) as e:
            lwq.lwq_attention_paged(p.cache(), p.q, out, 8, p.scale)
        assert e.value.status == lwq.LWQ_ERR_WORKSPACE_TOO_SMALL
        lwq.lwq_shutdown()
        with pytest.raises(lwq.LwqError) as e:
            lwq.lwq_attention_paged(p.cache(), p.q, out, 8, p.scale)
        assert e.value.status == lwq.LWQ_ERR_NOT_INITIALIZED
        exact = torch.full((need,), 0xFF, dtype=torch.uint8, device=dev)
        lwq.lwq_init(exact, need)
        check_attention(p, causal=False)
    finally:
        torch.cuda.synchronize(dev)
        lwq.lwq_init(_ARENA[0], WS_BYTES)


def test_tensors_that_do_not_fit_are_refused(dev):
    """int64 lengths, a strided query, an output of the other type or too small: refused before any launch."""
    p = Problem(dev, "f16", [30, 5], 4, 2, 64, 16, seed=1)
    f16, f32 = torch.zeros((2, 4, 64), dtype=torch.float16, device=dev), torch.zeros((2, 4, 64), device=dev)
    p.lens_d = p.lens_d.long()
    with pytest.raises(ValueError):
        p.cache()
    p.lens_d = p.lens_d.int()
    cache = p.cache()
    with pytest.raises(ValueError):
        lwq.lwq_attention_paged(cache, p.q, f16, 4, p.scale)
    with pytest.raises(ValueError):
        lwq.lwq_attention_paged(cache, p.q, f32, 4, p.scale, flags=lwq.LWQ_FLAG_OUT16)
    with pytest.raises(ValueError):
        lwq.lwq_attention_paged(cache, p.q, f32[:1], 4, p.scale)
    with pytest.raises(ValueError):
        lwq.lwq_attention_paged(cache, p.q.transpose(0, 1), f32, 4, p.scale)
    with pytest.raises(ValueError):
        lwq.lwq_kv_append(cache, None, lwq.LWQ_ACT_F32, f16, 512, f16, 512, f16, 512, f16, 2, 4)
    with pytest.raises(lwq.LwqError) as e:
        lwq.lwq_attention_paged(cache, p.q, p.q, 4, p.scale, flags=lwq.LWQ_FLAG_OUT16)
    assert e.value.status == lwq.LWQ_ERR_INVALID_ARG


def test_two_captured_graphs_in_turn(dev):
    """Two batches' decode steps, captured apart, share the workspace: replayed one after the other on one stream."""
    ps = [Problem(dev, "f16", [700, 3, 0], 8, 2, 64, 16, prefix=90, seed=1), Problem(dev, "f16", [4000], 8, 2, 64, 32, seed=2)]
    s = torch.cuda.Stream(dev)
    outs, graphs = [torch.zeros((p.B, 8, 64), device=dev) for p in ps], []
    for p, out in zip(ps, outs):
        cache = p.cache()
        lwq.lwq_attention_paged(cache, p.q, out, 8, p.scale, stream=s)
        s.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            lwq.lwq_attention_paged(cache, p.q, out, 8, p.scale, stream=s)
        out.zero_()
    torch.cuda.synchronize(dev)
    with torch.cuda.stream(s):
        for _ in range(3):
            for g in graphs:
                g.replay()
    torch.cuda.synchronize(dev)
    for p, out in zip(ps, outs):
        assert_attention(p, out, False)
    graphs.clear()


def test_prefill_no_live_token(dev):
    """Every sequence of a captured batch without a new token, keys split or not: nothing is written."""
    p = Problem(dev, "f16", [4000, 900], 8, 2, 64, 16, new=[0, 0], seed=1)
    for T in (1, 3000):
        out = torch.full((T, 8, 64), 5.0, device=dev)
        q = torch.zeros((T, 8, 64), dtype=torch.float16, device=dev)
        lwq.lwq_attention_prefill(p.cache(), q, out, p.cu_d, T, 8, p.scale)
        torch.cuda.synchronize(dev)
        assert (out == 5.0).all()
    assert lwq.lwq_get_device_error() == lwq.LWQ_OK


# ------------------------------------------------------------ a run of them all
def test_layer_prompt_then_decode(dev):
    """One attention layer as a server runs it: quantized qkv projection, append, prefill, quantized output
    projection for two ragged prompts; then two decode steps.  Each call's output against the oracles, on the
    inputs that it was given."""
    H, Hkv, D, K = 8, 2, 64, 512
    N = (H + 2 * Hkv) * D
    new = [70, 33]
    p = Problem(dev, "f16", new, H, Hkv, D, 16, new=new, seed=3, max_pages=6, spare=8)
    used = set(p.tables_h.flatten().tolist())
    free = [i for i in range(p.num_pages) if i not in used]
    for b in range(2):
        for i in range(6):
            if p.tables_h[b, i] < 0:
                p.tables_h[b, i] = free.pop(0) if free else 0
    p.tables.copy_(p.tables_h)
    Wqkv, _ = inputs.make_problem("q4_k", "f32", 1, N, K, seed=1)
    Wo, _ = inputs.make_problem("q8_0", "f32", 1, K, H * D, seed=2)
    Wqkv_d, Wo_d = to_device(Wqkv, dev), to_device(Wo, dev)
    fq, fo = lwq.fmt_code("q4_k", "f16"), lwq.fmt_code("q8_0", "f16")
    rope = lwq.lwq_rope_init(D)
    g = torch.Generator().manual_seed(4)
    cu = p.cu_d
    for step in range(3):
        T = sum(new) if step == 0 else 2
        p.new, p.T = (new, T) if step == 0 else ([1, 1], 2)
        p.cu = [0, new[0], sum(new)] if step == 0 else [0, 1, 2]
        p.lens = [n + step for n in new]
        p.lens_d.copy_(torch.tensor(p.lens, dtype=torch.int32))
        x = (0.02 * torch.randn((T, K), generator=g)).half().to(dev)
        y = torch.zeros((T, N), device=dev)
        lwq.lwq_matmul(fq, Wqkv_d, x, y, T, N, K)
        q = torch.zeros((T, H, D), dtype=torch.float16, device=dev)
        lwq.lwq_kv_append(p.cache(), rope, lwq.LWQ_ACT_F32, y, N, y[:, H * D:], N, y[:, (H + Hkv) * D:], N, q, T, H,
                          cu_tokens=cu if step == 0 else None)
        o = torch.zeros((T, H, D), dtype=torch.float16, device=dev)
        if step == 0:
            lwq.lwq_attention_prefill(p.cache(), q, o, cu, T, H, p.scale, flags=lwq.LWQ_FLAG_OUT16)
        else:
            lwq.lwq_attention_paged(p.cache(), q, o, H, p.scale, flags=lwq.LWQ_FLAG_OUT16)
        z = torch.zeros((T, K), device=dev)
        lwq.lwq_matmul(fo, Wo_d, o, z, T, K, H * D)
        torch.cuda.synchronize(dev)
        y_ref, den = oracle.matmul("q4_k", Wqkv, x.cpu().numpy(), act="f16")
        assert oracle.normalised_error(y.cpu().numpy(), y_ref, den) <= 5e-3
        place = [n - m + i for n, m in zip(p.lens, p.new) for i in range(m)]
        eq, ek, _ = expected_append(p, y, torch.tensor([place]), dict(rot=D, layout="half", base=10000.0))
        assert float(((q.double() - eq).abs() / (eq.abs() + 1e-3)).max()) < 2.0 ** -10
        p.q = q
        assert_attention(p, o, True, out16=True)
        z_ref, den = oracle.matmul("q8_0", Wo, o.view(T, -1).cpu().numpy(), act="f16")
        assert oracle.normalised_error(z.cpu().numpy(), z_ref, den) <= 5e-3
