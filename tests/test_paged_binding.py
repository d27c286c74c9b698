"""The binding's checks of the tensors that the paged-cache calls are given: element type, extent, device.  Every call
here is refused before the library is entered; the tensors only say that they are on a GPU."""

import pytest
import torch

import block_quantized_matmul_lwq_b200 as lwq
from block_quantized_matmul_lwq_b200 import build as lwq_build

P = 0x10000      # a pointer given as a number is taken as it is


@pytest.fixture(scope="module", autouse=True)
def built():
    lwq_build.build()


class OnGpu:
    """A host tensor that answers for one on cuda:index."""

    def __init__(self, t, index=0):
        self.t, self.index = t, index

    is_cuda = True
    device = "cuda (claimed)"

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


def gpu(shape, dtype, index=0):
    return OnGpu(torch.zeros(shape, dtype=dtype), index)


def cache(act=lwq.LWQ_ACT_F16, **kw):
    a = dict(k=P, v=P, tables=P, lens=P, prefix=None, prefix_len=0)
    a.update(kw)
    k, v, tables, lens = (a.pop(n) for n in ("k", "v", "tables", "lens"))
    return lwq.lwq_paged(act, k, v, tables, lens, B=3, Hkv=2, D=64, page=16, max_pages=4, num_pages=9, **a)


SHAPE = (9, 2, 16, 64)


@pytest.mark.parametrize("kw", [
    dict(k=gpu(SHAPE, torch.bfloat16)), dict(v=gpu(SHAPE, torch.bfloat16)), dict(v=gpu(SHAPE, torch.float32)),
    dict(tables=gpu((3, 4), torch.float32)), dict(lens=gpu(3, torch.float32)), dict(lens=gpu(3, torch.int64)),
    dict(lens=gpu(3, torch.int16)), dict(prefix=gpu(2, torch.float32), prefix_len=20),
    dict(act=lwq.LWQ_ACT_BF16, k=gpu(SHAPE, torch.float16)),
])
def test_caches_of_another_type(kw):
    with pytest.raises(ValueError):
        cache(**kw)


def test_raw_bits_are_taken():
    """16-bit integers hold the bits of either type."""
    for act in (lwq.LWQ_ACT_F16, lwq.LWQ_ACT_BF16):
        cache(act, k=gpu(SHAPE, torch.int16), v=gpu(SHAPE, torch.uint16))


@pytest.mark.parametrize("act,wrong", [(lwq.LWQ_ACT_F16, torch.bfloat16), (lwq.LWQ_ACT_BF16, torch.float16)])
def test_attention_types(act, wrong):
    c, w, f32, i32 = cache(act), gpu((3, 4, 64), wrong), gpu((3, 4, 64), torch.float32), gpu((3, 4, 64), torch.int32)
    for q, out, flags in ((w, f32, 0), (P, w, lwq.LWQ_FLAG_OUT16), (P, i32, 0)):
        with pytest.raises(ValueError):
            lwq.lwq_attention_paged(c, q, out, 4, 0.1, flags=flags)
        with pytest.raises(ValueError):
            lwq.lwq_attention_prefill(c, q, out, None, 3, 4, 0.1, flags=flags)
    with pytest.raises(ValueError):
        lwq.lwq_attention_prefill(c, P, P, gpu(4, torch.float32), 3, 4, 0.1)


N = 512       # (4 + 2 * 2) heads of 64


def append(**kw):
    a = dict(src=lwq.LWQ_ACT_F32, q=P, ldq=N, k=P, ldk=N, v=P, ldv=N, q_out=P, cu=None, pos=None)
    a.update(kw)
    lwq.lwq_kv_append(cache(), lwq.lwq_rope_init(64, sections=[16, 16]), a["src"], a["q"], a["ldq"], a["k"], a["ldk"],
                      a["v"], a["ldv"], a["q_out"], 3, 4, cu_tokens=a["cu"], positions=a["pos"])


def test_append_types():
    f16, b16, i32 = (gpu((3, N), t) for t in (torch.float16, torch.bfloat16, torch.int32))
    for bad in (f16, b16, i32):
        for name in ("q", "k", "v"):
            with pytest.raises(ValueError):
                append(**{name: bad})
    for name in ("q", "k", "v"):
        with pytest.raises(ValueError):
            append(src=lwq.LWQ_ACT_BF16, **{name: f16})
    for bad in (b16, gpu((3, N), torch.float32)):
        with pytest.raises(ValueError):
            append(q_out=bad)


def test_append_rows_that_end_early():
    """The last of T rows, ld apart, has to end within the tensor's memory: one element less is refused."""
    x = torch.zeros(3 * N)
    for name, first, width in (("q", 0, 256), ("k", 256, 128), ("v", 384, 128)):
        whole = torch.zeros(first + 2 * N + width)
        with pytest.raises(ValueError):
            append(**{name: OnGpu(whole[:-1].clone()[first:])})
        with pytest.raises(ValueError):
            append(**{name: OnGpu(x[first:]), "ld" + name: N + 400})
        with pytest.raises(ValueError):
            append(**{name: OnGpu(torch.zeros(2, N)[:, first:])})
        # enough: the next argument's refusal is the one met
        with pytest.raises(ValueError, match="positions"):
            append(**{name: OnGpu(whole[first:])}, pos=gpu(5, torch.int32))
        with pytest.raises(ValueError, match="positions"):
            append(**{name: OnGpu(x.view(3, N)[:, first:])}, pos=gpu(5, torch.int32))


@pytest.mark.parametrize("cu", [gpu(3, torch.int32), gpu(4, torch.float32), gpu(4, torch.int64),
                                OnGpu(torch.zeros(8, dtype=torch.int32)[::2])])
def test_append_offsets(cu):
    """B + 1 of them, in one piece."""
    with pytest.raises(ValueError, match="cu_tokens"):
        append(cu=cu)


def test_every_tensor_is_on_the_caches_device():
    c = cache(k=gpu(SHAPE, torch.float16, 1), v=gpu(SHAPE, torch.float16, 1))
    f16, f32, cu = gpu((3, 4, 64), torch.float16), gpu((3, 4, 64), torch.float32), gpu(4, torch.int32)
    with pytest.raises(ValueError):
        cache(k=gpu(SHAPE, torch.float16, 1), lens=gpu(3, torch.int32, 0))
    for q, out in ((f16, P), (P, f32)):
        with pytest.raises(ValueError):
            lwq.lwq_attention_paged(c, q, out, 4, 0.1)
    with pytest.raises(ValueError, match="cu_tokens"):
        lwq.lwq_attention_prefill(c, P, P, cu, 3, 4, 0.1)
    x = gpu((3, N), torch.float32)
    for kw in (dict(q=x), dict(k=x), dict(v=x), dict(q_out=f16), dict(cu=cu), dict(pos=gpu(6, torch.int32))):
        a = dict(q=P, k=P, v=P, q_out=P, cu=None, pos=None)
        a.update(kw)
        with pytest.raises(ValueError):
            lwq.lwq_kv_append(c, lwq.lwq_rope_init(64, sections=[16, 16]), lwq.LWQ_ACT_F32, a["q"], N, a["k"], N, a["v"], N,
                              a["q_out"], 3, 4, cu_tokens=a["cu"], positions=a["pos"])


def test_a_copied_cache_is_a_cache():
    """Its tensors are not known, so only the call's own are looked at."""
    c = lwq.lwq_paged.from_buffer_copy(cache(k=gpu(SHAPE, torch.float16)))
    with pytest.raises(ValueError):
        lwq.lwq_attention_paged(c, gpu((3, 4, 64), torch.bfloat16), P, 4, 0.1)
    with pytest.raises(lwq.LwqError) as e:
        lwq.lwq_attention_paged(c, P, P, 5, 0.1)
    assert e.value.status == lwq.LWQ_ERR_INVALID_ARG
