"""Host-side checks of the paged-cache entry points: refusals and the rotation table.  No call here reaches a GPU
(every checked call returns before any device work)."""

import math

import pytest

import block_quantized_matmul_lwq_b200 as lwq
from block_quantized_matmul_lwq_b200 import build as lwq_build


@pytest.fixture(scope="module", autouse=True)
def built():
    lwq_build.build()


FAKE = 0x10000   # 16-byte aligned host integers; never dereferenced by the checks below
QOUT = 0x40000000


def cache(**kw):
    a = dict(act=lwq.LWQ_ACT_F16, k=FAKE, v=FAKE, tables=FAKE, lens=FAKE, B=2, Hkv=2, D=64, page=16, max_pages=4,
             num_pages=9, prefix=None, prefix_len=0)
    a.update(kw)
    act, k, v, tables, lens = (a.pop(n) for n in ("act", "k", "v", "tables", "lens"))
    return lwq.lwq_paged(act, k, v, tables, lens, **a)


BAD_CACHES = [
    (dict(B=0), 1), (dict(Hkv=0), 1), (dict(max_pages=0), 1), (dict(num_pages=-1), 1), (dict(prefix_len=-1), 1),
    (dict(prefix_len=5), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(tables=None), 1), (dict(lens=None), 1),
    (dict(Hkv=3), 1),                                   # 4 heads over 3
    (dict(act=lwq.LWQ_ACT_F32), 2), (dict(act=7), 2), (dict(D=96), 2), (dict(page=8), 2), (dict(page=24), 2),
    (dict(page=512), 2), (dict(num_pages=1 << 30), 2), (dict(max_pages=1 << 30), 2), (dict(B=70000), 2),
    (dict(k=FAKE + 8), 3), (dict(v=FAKE + 2), 3), (dict(tables=FAKE + 2), 3), (dict(lens=FAKE + 1), 3),
    (dict(prefix=FAKE + 2, prefix_len=4), 3),
]


def status(call, *args, **kw):
    try:
        call(*args, **kw)
    except lwq.LwqError as e:
        return e.status
    return 0


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_caches(kw, code):
    c = cache(**kw)
    if "B" in kw and kw["B"] <= 0:
        T = 1
    else:
        T = c.B
    assert status(lwq.lwq_kv_append, c, None, lwq.LWQ_ACT_F16, FAKE, 512, FAKE, 512, FAKE, 512, QOUT, T, 4) == code
    assert status(lwq.lwq_attention_paged, c, FAKE, FAKE, 4, 0.1) == code
    assert status(lwq.lwq_attention_prefill, c, FAKE, FAKE, FAKE, 5, 4, 0.1) == code


def test_heads_per_kv_head():
    assert status(lwq.lwq_attention_paged, cache(Hkv=1), FAKE, FAKE, 17, 0.1) == lwq.LWQ_ERR_UNSUPPORTED
    assert status(lwq.lwq_attention_paged, cache(Hkv=1), FAKE, FAKE, 0, 0.1) == lwq.LWQ_ERR_INVALID_ARG


@pytest.mark.parametrize("args,code", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(flags=1), 2), (dict(flags=lwq.LWQ_FLAG_OVERLAP), 2), (dict(q=FAKE + 8), 3), (dict(out=FAKE + 4), 3),
])
def test_bad_attention_arguments(args, code):
    a = dict(q=FAKE, out=FAKE, scale=0.1, flags=0)
    a.update(args)
    assert status(lwq.lwq_attention_paged, cache(), a["q"], a["out"], 4, a["scale"], flags=a["flags"]) == code
    assert status(lwq.lwq_attention_prefill, cache(), a["q"], a["out"], FAKE, 5, 4, a["scale"],
                  flags=a["flags"]) == code


def test_out_may_not_overlap_q():
    """No in-place form, whichever type out has: q is read by CTAs that others do not wait for."""
    n = 2 * 4 * 64                                      # B x H x D
    for flags, es in ((0, 4), (lwq.LWQ_FLAG_OUT16, 2)):
        for out in (FAKE, FAKE + 2 * n - 16, FAKE - es * n + 16):
            assert status(lwq.lwq_attention_paged, cache(), FAKE, out, 4, 0.1, flags=flags) == lwq.LWQ_ERR_INVALID_ARG
            assert status(lwq.lwq_attention_prefill, cache(), FAKE, out, None, 2, 4, 0.1,
                          flags=flags) == lwq.LWQ_ERR_INVALID_ARG


def test_scale_past_the_range_of_the_exponents():
    """scale log2(e) has to be finite, as the kernels take powers of two."""
    assert status(lwq.lwq_attention_paged, cache(), FAKE, QOUT, 4, 3e38) == lwq.LWQ_ERR_INVALID_ARG


def test_tensors_on_the_host_are_refused():
    torch = pytest.importorskip("torch")
    t32, t16 = torch.zeros(4096), torch.zeros(4096, dtype=torch.float16)
    with pytest.raises(ValueError):
        cache(k=t16)
    with pytest.raises(ValueError):
        cache(lens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        lwq.lwq_attention_paged(cache(), t16, QOUT, 4, 0.1)
    with pytest.raises(ValueError):
        lwq.lwq_attention_prefill(cache(), FAKE, t32, FAKE, 2, 4, 0.1)
    with pytest.raises(ValueError):
        lwq.lwq_kv_append(cache(), None, lwq.LWQ_ACT_F32, FAKE, 512, t32, 512, FAKE, 512, QOUT, 2, 4)


def test_a_copied_rotation_is_the_rotation():
    rope = lwq.lwq_rope.from_buffer_copy(lwq.lwq_rope_init(128))
    assert status(lwq.lwq_kv_append, cache(), rope, lwq.LWQ_ACT_F16, FAKE, 512, FAKE, 512, FAKE, 512, QOUT, 2,
                  4) == lwq.LWQ_ERR_UNSUPPORTED        # looked at: wider than the head


def test_prefill_counts():
    assert status(lwq.lwq_attention_prefill, cache(), FAKE, FAKE, FAKE, 0, 4, 0.1) == lwq.LWQ_ERR_INVALID_ARG
    assert status(lwq.lwq_attention_prefill, cache(), FAKE, FAKE, None, 3, 4, 0.1) == lwq.LWQ_ERR_INVALID_ARG
    assert status(lwq.lwq_attention_prefill, cache(), FAKE, FAKE, FAKE + 2, 5, 4, 0.1) == lwq.LWQ_ERR_MISALIGNED
    assert status(lwq.lwq_attention_prefill, cache(), FAKE, FAKE, FAKE, 1 << 30, 4, 0.1) == lwq.LWQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("args,code", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(q=None), 1), (dict(q_out=None), 1), (dict(T=0), 1),
    (dict(T=3), 1),                                     # without cu_tokens: one token per sequence
    (dict(ldq=248), 1), (dict(ldk=120), 1), (dict(ldv=120), 1),
    (dict(q_out=FAKE), 1), (dict(q_out=FAKE + 512), 1),   # over the inputs
    (dict(src=lwq.LWQ_Q4_0), 2), (dict(src=0x300), 2), (dict(ldk=1 << 50), 2),
    (dict(q=FAKE + 4), 3), (dict(k=FAKE + 8), 3), (dict(v=FAKE + 2), 3), (dict(q_out=QOUT + 8), 3),
    (dict(ldq=516), 3), (dict(ldk=516), 3), (dict(ldv=514), 3), (dict(cu=FAKE + 2), 3), (dict(pos=FAKE + 2), 3),
])
def test_bad_append_arguments(args, code):
    a = dict(src=lwq.LWQ_ACT_F16, q=FAKE, ldq=512, k=FAKE, ldk=512, v=FAKE, ldv=512, q_out=QOUT, T=2, cu=None, pos=None)
    a.update(args)
    assert status(lwq.lwq_kv_append, cache(), None, a["src"], a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"],
                  a["q_out"], a["T"], 4, cu_tokens=a["cu"], positions=a["pos"]) == code


def test_append_checks_the_rotation():
    def with_rope(rope):
        return status(lwq.lwq_kv_append, cache(), rope, lwq.LWQ_ACT_F16, FAKE, 512, FAKE, 512, FAKE, 512, QOUT, 2, 4)

    assert with_rope(lwq.lwq_rope_init(128)) == lwq.LWQ_ERR_UNSUPPORTED        # wider than the head
    assert with_rope(lwq.lwq_rope()) == lwq.LWQ_ERR_UNSUPPORTED                # never initialised
    rope = lwq.lwq_rope_init(64)
    rope.axis[3] = 1
    assert with_rope(rope) == lwq.LWQ_ERR_INVALID_ARG                          # an axis that there is not


@pytest.mark.parametrize("kw,code", [
    (dict(rot_dim=0), 2), (dict(rot_dim=24), 2), (dict(rot_dim=144), 2), (dict(rot_dim=64, layout=2), 2),
    (dict(rot_dim=64, base=0.0), 1), (dict(rot_dim=64, base=-1.0), 1), (dict(rot_dim=64, base=float("nan")), 1),
    (dict(rot_dim=64, sections=[16, 8]), 1), (dict(rot_dim=64, sections=[32, 8]), 1),
    (dict(rot_dim=64, sections=[40, -8]), 1), (dict(rot_dim=64, sections=[8, 8, 8, 4, 4]), 2),
    (dict(rot_dim=16, inv_freq=[1.0] * 7 + [float("inf")]), 1), (dict(rot_dim=16, inv_freq=[1e9] * 8), 1),
])
def test_bad_rotations(kw, code):
    assert status(lwq.lwq_rope_init, **kw) == code


def test_inv_freq_needs_every_pair():
    with pytest.raises(ValueError):
        lwq.lwq_rope_init(64, inv_freq=[1.0] * 31)


@pytest.mark.parametrize("rot,base", [(64, 10000.0), (128, 1e6), (16, 500000.0)])
def test_rotation_table(rot, base):
    """turn[i] 2^-64 is base^(-2 i / rot) / (2 pi) modulo 1: to the table's unit of 2^-64 turns, beside what the
    doubles here are off by (an exponent below 32 in size, rounded three times: 2^-47 of the value)."""
    r = lwq.lwq_rope_init(rot, base=base)
    assert (r.rot_dim, r.layout, r.axes) == (rot, lwq.LWQ_ROPE_HALF, 1)
    for i in range(rot // 2):
        want = math.exp(-2 * i / rot * math.log(base)) / (2 * math.pi)
        assert abs(r.turn[i] * 2.0 ** -64 - want) <= 2.0 ** -64 + 2.0 ** -47 * want
        assert r.axis[i] == 0


def test_rotation_axes_and_frequencies():
    r = lwq.lwq_rope_init(32, inv_freq=[-1.0, 0.0, 7.5] + [0.25] * 13, sections=[2, 0, 5, 9], layout=lwq.LWQ_ROPE_PAIRS)
    assert list(r.axis[:16]) == [0] * 2 + [2] * 5 + [3] * 9
    assert abs(r.turn[0] * 2.0 ** -64 - (1 - 1 / (2 * math.pi))) < 1e-15      # a negative frequency turns back
    assert r.turn[1] == 0
    assert abs(r.turn[2] * 2.0 ** -64 - (7.5 / (2 * math.pi) - 1)) < 1e-15    # only the part of a turn counts


def test_workspace_sizes():
    """Sizes come from the description alone and do not depend on its pointers; 0 for what is refused."""
    c = cache(k=None, v=None, tables=None, lens=None)
    assert lwq.lwq_attention_paged_workspace_size(c, 4) > 0
    assert lwq.lwq_attention_prefill_workspace_size(c, 100, 4) > 0
    assert lwq.lwq_attention_paged_workspace_size(cache(D=96), 4) == 0
    assert lwq.lwq_attention_paged_workspace_size(cache(), 5) == 0
    assert lwq.lwq_attention_prefill_workspace_size(cache(), 0, 4) == 0
    assert lwq.lwq_status_string(lwq.LWQ_ERR_BAD_PAGE) != lwq.lwq_status_string(99)
