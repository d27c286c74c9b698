// Host side of the paged key/value cache: argument checks, work division and
// launches (see include/lwq.h).  Included by lwq_api.cu: the library is one
// translation unit, with one copy of the device error word.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "../../include/lwq.h"
#include "lwq_paged.cuh"
#include "lwq_paged_decode.cuh"
#include "lwq_paged_tile.cuh"

namespace lwq {
namespace {

constexpr long kMaxIndex = 0x7fffffffl;

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Sizes and types of the cache description alone (the workspace sizes need no pointers).
int paged_sizes(const lwq_paged *c, int H) {
    if (!c || c->B <= 0 || c->Hkv <= 0 || c->D <= 0 || c->page <= 0 || c->max_pages <= 0 || c->num_pages <= 0 ||
        c->prefix_len < 0 || H <= 0)
        return LWQ_ERR_INVALID_ARG;
    if (c->dtype != LWQ_ACT_F16 && c->dtype != LWQ_ACT_BF16) return LWQ_ERR_UNSUPPORTED;
    if (c->D != 64 && c->D != 128) return LWQ_ERR_UNSUPPORTED;
    if (c->page < 16 || c->page > 256 || (c->page & (c->page - 1))) return LWQ_ERR_UNSUPPORTED;
    if (H % c->Hkv) return LWQ_ERR_INVALID_ARG;
    if (H / c->Hkv > 16) return LWQ_ERR_UNSUPPORTED;
    // token rows of the cache and places of a sequence are 32-bit numbers in the kernels
    if ((double)c->num_pages * c->Hkv * c->page > (double)kMaxIndex) return LWQ_ERR_UNSUPPORTED;
    if ((double)c->max_pages * c->page + c->prefix_len > (double)(kMaxIndex - 1024)) return LWQ_ERR_UNSUPPORTED;
    if (c->B > 65535 || c->Hkv > 65535) return LWQ_ERR_UNSUPPORTED;
    return LWQ_OK;
}

int paged_pointers(const lwq_paged *c) {
    if (!c->k || !c->v || !c->tables || !c->lens || (c->prefix_len > 0 && !c->prefix)) return LWQ_ERR_INVALID_ARG;
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned4(c->tables) || !aligned4(c->lens) || !aligned4(c->prefix))
        return LWQ_ERR_MISALIGNED;
    return LWQ_OK;
}

PagedArgs paged_args(const lwq_paged *c) {
    PagedArgs p;
    p.k = static_cast<uint16_t *>(c->k);
    p.v = static_cast<uint16_t *>(c->v);
    p.tables = c->tables;
    p.lens = c->lens;
    p.prefix = c->prefix;
    p.prefix_len = c->prefix_len;
    p.B = c->B;
    p.Hkv = c->Hkv;
    p.page = c->page;
    p.page_shift = 0;
    while ((1 << p.page_shift) < c->page) ++p.page_shift;
    p.max_pages = c->max_pages;
    p.num_pages = c->num_pages;
    return p;
}

// [a, a + an) and [b, b + bn) share a byte
bool overlap(const void *a, size_t an, const void *b, size_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + bn && y < x + an;
}

// [a, a + an) shares a byte with the cache's pages
bool overlaps_cache(const lwq_paged *c, const void *a, size_t an) {
    const size_t n = (size_t)c->num_pages * c->Hkv * c->page * c->D * 2;
    return overlap(a, an, c->k, n) || overlap(a, an, c->v, n);
}

int rope_check(const lwq_rope *r, int D) {
    if (r->rot_dim < 16 || r->rot_dim % 16 || r->rot_dim > D) return LWQ_ERR_UNSUPPORTED;
    if (r->layout != LWQ_ROPE_HALF && r->layout != LWQ_ROPE_PAIRS) return LWQ_ERR_UNSUPPORTED;
    if (r->axes < 1 || r->axes > 4) return LWQ_ERR_UNSUPPORTED;
    for (int i = 0; i < r->rot_dim / 2; ++i)
        if (r->axis[i] >= r->axes) return LWQ_ERR_INVALID_ARG;
    return LWQ_OK;
}

// f / (2 pi) modulo 1 in units of 2^-64, rounded to nearest, |f| below 2^63: all 64 bits of f's significand times 192
// bits of 1 / (2 pi) in integers (a quotient in floating point would lose below what the whole turns leave).
uint64_t turn_of(long double f) {
    constexpr uint64_t inv[3] = {0x36d8a5664f10e410ull, 0x7f09d5f47d4d3770ull, 0x28be60db9391054aull};   // lowest first
    int e;
    const uint64_t m = (uint64_t)ldexpl(frexpl(fabsl(f), &e), 64);   // |f| = m 2^(e - 64)
    uint64_t p[5] = {};                                              // m / (2 pi) in units of 2^-192
    unsigned __int128 carry = 0;
    for (int i = 0; i < 3; ++i) {
        carry += (unsigned __int128)m * inv[i];
        p[i] = (uint64_t)carry;
        carry >>= 64;
    }
    p[3] = (uint64_t)carry;
    const int at = 192 - e;          // the bit of p that weighs 2^-64 turns
    auto bits = [&](int k) {         // 64 bits of p from bit k on
        const int w = k / 64, b = k % 64;
        return w > 3 ? 0 : b ? p[w] >> b | p[w + 1] << (64 - b) : p[w];
    };
    const uint64_t u = bits(at) + (bits(at - 1) & 1);
    return f < 0 ? 0 - u : u;
}

template <int ST, int XT>
cudaError_t launch_append(int D, const AppendArgs &a, const lwq_rope &rope, cudaStream_t st) {
    // a block per token (several where its rows need more than 8 warps): never less than the 64 threads of its pairs,
    // as k and v take a warp each
    const int units = a.uq + 2 * a.uk, warps = units < APPEND_WARPS ? units : APPEND_WARPS;
    const dim3 grid((unsigned)a.T, (unsigned)((units + APPEND_WARPS - 1) / APPEND_WARPS));
    if (D == 64)
        kv_append_kernel<ST, XT, 64><<<grid, warps * 32, 0, st>>>(a, rope);
    else
        kv_append_kernel<ST, XT, 128><<<grid, warps * 32, 0, st>>>(a, rope);
    return cudaGetLastError();
}
template <int ST>
cudaError_t launch_append_xt(int dtype, int D, const AppendArgs &a, const lwq_rope &rope, cudaStream_t st) {
    return dtype == LWQ_ACT_F16 ? launch_append<ST, X_F16>(D, a, rope, st)
                                : launch_append<ST, X_BF16>(D, a, rope, st);
}

// The checks that both attention calls make, and the kernels' view of the arguments.
int paged_attn_args(const lwq_paged *c, int flags, const void *q, void *out, const int32_t *cu, int T, int H,
                    float scale, PagedAttnArgs *a) {
    int rc = paged_sizes(c, H);
    if (rc) return rc;
    if (T <= 0 || !q || !out || (!cu && T != c->B) || !isfinite(scale)) return LWQ_ERR_INVALID_ARG;
    if ((rc = paged_pointers(c))) return rc;
    if (flags & ~LWQ_FLAG_OUT16) return LWQ_ERR_UNSUPPORTED;
    if ((double)T * H > (double)kMaxIndex) return LWQ_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(out) || !aligned4(cu)) return LWQ_ERR_MISALIGNED;
    a->c = paged_args(c);
    a->q = static_cast<const uint16_t *>(q);
    a->out = out;
    a->cu = cu;
    a->T = T;
    a->H = H;
    a->G = H / c->Hkv;
    a->out16 = (flags & LWQ_FLAG_OUT16) ? 1 : 0;
    a->qscale = scale * 1.4426950408889634f;   // log2(e): the kernels take exponentials as exp2
    if (!isfinite(a->qscale)) return LWQ_ERR_INVALID_ARG;
    const size_t n = (size_t)T * H * c->D;
    if (overlap(q, 2 * n, out, (a->out16 ? 2 : 4) * n) || overlaps_cache(c, out, (a->out16 ? 2 : 4) * n))
        return LWQ_ERR_INVALID_ARG;
    return LWQ_OK;
}

int paged_workspace(int dev, size_t need, void **ws) {
    *ws = nullptr;
    if (need == 0) return LWQ_OK;
    if (!g_dev[dev].registered) return LWQ_ERR_NOT_INITIALIZED;
    if (g_dev[dev].ws_bytes < need) return LWQ_ERR_WORKSPACE_TOO_SMALL;
    *ws = g_dev[dev].ws;
    return LWQ_OK;
}

// ------------------------------------------------------------------ decode
constexpr int kDecodeCtasPerSm = 2;

template <int XT, int D, int NG, int PARTS>
cudaError_t launch_paged_decode(const PagedPrefixArgs &k, cudaStream_t st) {
    auto kern = paged_decode_kernel<XT, D, NG, PARTS>;
    constexpr size_t smem = PagedDecodeSmem<D, NG>::TOTAL;
    const PagedDecodeArgs &d = k.d;
    cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kern), smem);
    if (e != cudaSuccess) return e;
    // behind a prefix's row tiles: a dependent launch, which starts as their CTAs end and waits for the last of them at
    // its own end
    if ((e = launch_k(kern, d.ctas, PD_WARPS * 32, smem, st, k.prefix != nullptr, d)) != cudaSuccess) return e;
    if (!k.prefix) {
        const int parts = combine_parts((long)d.a.c.B * d.a.c.Hkv, d.a.G, d.ctas), n = d.a.G * D / parts;
        const int threads = n >= PC_THREADS ? PC_THREADS : 2 * n <= PC_THREADS ? 2 * n : n;   // two groups where they fit
        return launch_k(paged_combine_kernel<XT, D>, d.ctas * parts, threads, 0, st, true, d, parts);
    }
    return launch_k(paged_prefix_combine_kernel<XT, D>, (int)(((long)d.a.c.B * d.a.H + 7) / 8), 256, 0, st, true, k);
}
template <int XT, int D, int PARTS>
cudaError_t launch_paged_decode_g(const PagedPrefixArgs &k, cudaStream_t st) {
    return k.d.a.G <= 8 ? launch_paged_decode<XT, D, 1, PARTS>(k, st) : launch_paged_decode<XT, D, 2, PARTS>(k, st);
}
// fp16's two parts of a probability hold 22 bits; bf16 takes a third part for an fp32 result
template <int D>
cudaError_t launch_paged_decode_x(int dtype, const PagedPrefixArgs &k, cudaStream_t st) {
    if (dtype == LWQ_ACT_F16) return launch_paged_decode_g<X_F16, D, 2>(k, st);
    return k.d.a.out16 ? launch_paged_decode_g<X_BF16, D, 2>(k, st) : launch_paged_decode_g<X_BF16, D, 3>(k, st);
}

// -------------------------------------------------------------- row tiles
template <int XT, int D, int PARTS>
int launch_paged_tile(const lwq_paged *c, PagedTileArgs &t, cudaStream_t st) {
    // three parts of a probability fit beside each other for 64 keys at a time
    constexpr int KT = PARTS == 3 ? 64 : 128;
    auto kern = paged_tile_kernel<XT, D, PARTS, KT>;
    constexpr size_t smem = TileSmem<D, KT>::TOTAL;
    const int brows = c->page < KT ? c->page : KT;
    CUtensorMap maps[2];
    for (int i = 0; i < 2; ++i) {
        MapReq r = map_req(i ? c->v : c->k, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, CU_TENSOR_MAP_SWIZZLE_128B);
        r.dims[0] = (cuuint64_t)D;
        r.dims[1] = (cuuint64_t)t.total_rows;
        r.strides[0] = (cuuint64_t)D * 2;
        r.box[0] = 64;
        r.box[1] = (cuuint32_t)brows;
        if (encode_cached(r, &maps[i])) return LWQ_ERR_CUDA;
    }
    if (ensure_smem(reinterpret_cast<const void *>(kern), smem) != cudaSuccess) return LWQ_ERR_CUDA;
    if (launch_k(kern, (int)(t.pairs * c->Hkv * t.splits), TILE_THREADS, smem, st, false, maps[0], maps[1], t) != cudaSuccess)
        return LWQ_ERR_CUDA;
    if (t.prefix_only || t.splits == 1) return LWQ_OK;
    return launch_k(paged_tile_combine_kernel<XT, D>, (int)(((long)t.a.T * t.a.H + 7) / 8), 256, 0, st, true, t) ==
                   cudaSuccess
               ? LWQ_OK
               : LWQ_ERR_CUDA;
}
// The parts of a probability: see the kernel's header.  A prefix's partial results go on to other sums in fp32, but a
// 16-bit result is no nearer for that.
template <int D>
int launch_paged_tile_x(const lwq_paged *c, PagedTileArgs &t, cudaStream_t st) {
    if (c->dtype == LWQ_ACT_F16)
        return t.a.out16 ? launch_paged_tile<X_F16, D, 1>(c, t, st) : launch_paged_tile<X_F16, D, 2>(c, t, st);
    return t.a.out16 ? launch_paged_tile<X_BF16, D, 1>(c, t, st) : launch_paged_tile<X_BF16, D, 3>(c, t, st);
}

PagedTileArgs paged_tile_args(const lwq_paged *c, const PagedAttnArgs &a, long pairs, int splits, float *part) {
    PagedTileArgs t;
    t.a = a;
    t.flip = a.qscale < 0.f;
    t.a.qscale = fabsf(a.qscale);
    // scale 0: a masked score stays -inf, any other becomes 0 (below 4, however large the product of query and key)
    if (t.a.qscale < FLT_MIN) t.a.qscale = FLT_MIN;
    t.part = part;
    t.splits = splits;
    t.pairs = pairs;
    t.prefix_only = 0;
    t.total_rows = c->num_pages * c->Hkv * c->page;
    t.timeout_ns = kTimeoutNs;
    return t;
}

// Pairs of row tiles that T tokens of at most B sequences can make, and into how many parts each pair's keys are cut:
// one when the pairs fill the GPU (a CTA per SM), else as many as do, but no part below one tile of 128 keys.
long tile_pairs(long T, int B, int G) { return T * G / PAIR_ROWS + (B < T ? B : T); }
int tile_splits(long pairs, int Hkv, long keys, int sms) {
    const long items = pairs * Hkv;
    long s = items >= sms ? 1 : sms / items;
    const long tiles = (keys + 127) / 128;
    if (s > tiles) s = tiles;
    return s < 1 ? 1 : (int)s;
}
size_t tile_part_bytes(long pairs, int Hkv, int splits, int D) {
    return (size_t)pairs * Hkv * splits * PAIR_ROWS * part_stride(D) * sizeof(float);
}

// The most bytes that up to `pairs` pairs take: fewer pairs are cut into more parts (whole: pairs that are not cut have
// partial results too).
size_t tile_part_most(long pairs, int Hkv, long keys, int sms, int D, bool whole) {
    size_t most = whole ? tile_part_bytes(pairs, Hkv, 1, D) : 0;
    for (long p = 1; p <= pairs && p * Hkv * 2 <= sms; ++p) {   // (beyond, tile_splits is 1)
        const size_t n = tile_part_bytes(p, Hkv, tile_splits(p, Hkv, keys, sms), D);
        if (n > most) most = n;
    }
    return most;
}

// How a prefill call is divided.
void prefill_plan(const lwq_paged *c, int T, int H, int sms, long *pairs, int *splits) {
    *pairs = tile_pairs(T, c->B, H / c->Hkv);
    *splits = tile_splits(*pairs, c->Hkv, (long)c->max_pages * c->page + c->prefix_len, sms);
}

// The parts of a decode call's workspace: the CTAs' slots and the list of pairs that several CTAs work on, then, with a
// prefix, one result per (sequence, head) and the prefix's partial results.
struct DecodeSpace {
    size_t slots, list, whole, prefix;
    long pairs;
    int splits;
    size_t total() const { return slots + list + whole + prefix; }
};
DecodeSpace decode_space(const lwq_paged *c, int H, int sms) {
    DecodeSpace s;
    const int G = H / c->Hkv;
    const size_t ps = part_stride(c->D) * sizeof(float);
    s.slots = (size_t)kDecodeCtasPerSm * sms * 2 * G * ps;
    s.list = (size_t)kDecodeCtasPerSm * sms * sizeof(int4);
    s.whole = s.prefix = 0;
    s.pairs = 0;
    s.splits = 0;
    if (c->prefix_len > 0) {
        s.whole = (size_t)c->B * H * ps;
        s.pairs = pairs_of(c->B, G);
        s.splits = tile_splits(s.pairs, c->Hkv, c->prefix_len, sms);
        s.prefix = tile_part_bytes(s.pairs, c->Hkv, s.splits, c->D);
    }
    return s;
}

}  // namespace
}  // namespace lwq

extern "C" {

int lwq_rope_init(lwq_rope *rope, int rot_dim, int layout, double base, const double *inv_freq, int axes,
                  const int *sections) {
    if (!rope || (!sections && axes != 1)) return LWQ_ERR_INVALID_ARG;
    if (rot_dim < 16 || rot_dim > 128 || rot_dim % 16 || axes < 1 || axes > 4 ||
        (layout != LWQ_ROPE_HALF && layout != LWQ_ROPE_PAIRS))
        return LWQ_ERR_UNSUPPORTED;
    if (!inv_freq && !(isfinite(base) && base > 0)) return LWQ_ERR_INVALID_ARG;
    const int half = rot_dim / 2;
    lwq_rope r;
    memset(&r, 0, sizeof(r));
    r.rot_dim = rot_dim;
    r.layout = layout;
    r.axes = axes;
    int at = 0;
    for (int a = 0; a < axes; ++a) {
        const int n = sections ? sections[a] : half;
        if (n < 0 || n > half - at) return LWQ_ERR_INVALID_ARG;
        for (int i = 0; i < n; ++i) r.axis[at++] = (uint8_t)a;
    }
    if (at != half) return LWQ_ERR_INVALID_ARG;
    for (int i = 0; i < half; ++i) {
        const long double f = inv_freq ? (long double)inv_freq[i] : powl((long double)base, -2.0L * i / rot_dim);
        if (!isfinite(f) || fabsl(f) > (inv_freq ? 1048576.0L : 256.0L)) return LWQ_ERR_INVALID_ARG;
        r.turn[i] = turn_of(f);
    }
    *rope = r;
    return LWQ_OK;
}

int lwq_kv_append(const lwq_paged *cache, const lwq_rope *rope, int src, const void *q, int64_t ldq, const void *k,
                  int64_t ldk, const void *v, int64_t ldv, void *q_out, const int32_t *cu_tokens,
                  const int32_t *positions, int T, int H, void *stream) {
    t_last_launches = 0;
    int rc = paged_sizes(cache, H);
    if (rc) return rc;
    if (T <= 0 || !k || !v || !q != !q_out || (!cu_tokens && T != cache->B)) return LWQ_ERR_INVALID_ARG;
    if ((rc = paged_pointers(cache))) return rc;
    const int D = cache->D;
    if (src != LWQ_ACT_F32 && src != LWQ_ACT_F16 && src != LWQ_ACT_BF16) return LWQ_ERR_UNSUPPORTED;
    if (rope && (rc = rope_check(rope, D))) return rc;
    if ((q && ldq < (int64_t)H * D) || ldk < (int64_t)cache->Hkv * D || ldv < (int64_t)cache->Hkv * D)
        return LWQ_ERR_INVALID_ARG;
    const int64_t es = src == LWQ_ACT_F32 ? 4 : 2, big = (int64_t)1 << 40;
    if ((q && ldq > big) || ldk > big || ldv > big) return LWQ_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned4(cu_tokens) ||
        !aligned4(positions) || (q && ldq * es % 16) || ldk * es % 16 || ldv * es % 16)
        return LWQ_ERR_MISALIGNED;
    if (q) {
        const size_t n = (size_t)T * H * D * 2;
        if (overlap(q_out, n, q, ((size_t)(T - 1) * ldq + (size_t)H * D) * es) ||
            overlap(q_out, n, k, ((size_t)(T - 1) * ldk + (size_t)cache->Hkv * D) * es) ||
            overlap(q_out, n, v, ((size_t)(T - 1) * ldv + (size_t)cache->Hkv * D) * es) || overlaps_cache(cache, q_out, n))
            return LWQ_ERR_INVALID_ARG;
    }
    int dev;
    if ((rc = current_device(&dev))) return rc;
    AppendArgs a;
    a.c = paged_args(cache);
    a.q = q;
    a.k = k;
    a.v = v;
    a.ldq = ldq;
    a.ldk = ldk;
    a.ldv = ldv;
    a.q_out = static_cast<uint16_t *>(q_out);
    a.cu = cu_tokens;
    a.positions = positions;
    a.T = T;
    a.H = H;
    const int per = APPEND_ITERS * (256 / D);   // heads per warp
    a.uq = q ? (H + per - 1) / per : 0;
    a.uk = (cache->Hkv + per - 1) / per;
    if ((a.uq + 2 * a.uk) / APPEND_WARPS >= 65535) return LWQ_ERR_UNSUPPORTED;
    a.rope = rope ? 1 : 0;
    a.pairs_layout = rope && rope->layout == LWQ_ROPE_PAIRS;
    lwq_rope r;
    if (rope)
        r = *rope;
    else
        memset(&r, 0, sizeof(r));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (src == LWQ_ACT_F32)
        e = launch_append_xt<X_F32>(cache->dtype, D, a, r, st);
    else if (src == LWQ_ACT_F16)
        e = launch_append_xt<X_F16>(cache->dtype, D, a, r, st);
    else
        e = launch_append_xt<X_BF16>(cache->dtype, D, a, r, st);
    if (e != cudaSuccess) return LWQ_ERR_CUDA;
    t_last_launches = 1;
    return LWQ_OK;
}

size_t lwq_attention_paged_workspace_size(const lwq_paged *cache, int H) {
    if (paged_sizes(cache, H)) return 0;
    int dev = 0, sms = 148;
    if (current_device(&dev) == LWQ_OK) sms = sm_count(dev);
    DecodeSpace s = decode_space(cache, H, sms);
    if (cache->prefix_len > 0) s.prefix = tile_part_most(s.pairs, cache->Hkv, cache->prefix_len, sms, cache->D, true);
    return s.total();
}

int lwq_attention_paged(const lwq_paged *cache, int flags, const void *q, void *out, int H, float scale,
                        void *stream) {
    t_last_launches = 0;
    PagedAttnArgs a;
    int rc = paged_attn_args(cache, flags, q, out, nullptr, cache ? cache->B : 0, H, scale, &a);
    if (rc) return rc;
    int dev;
    if ((rc = current_device(&dev))) return rc;
    const DecodeSpace sp = decode_space(cache, H, sm_count(dev));
    void *ws;
    if ((rc = paged_workspace(dev, sp.total(), &ws))) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    PagedPrefixArgs k;
    PagedDecodeArgs &d = k.d;
    d.a = a;
    d.slots = static_cast<float *>(ws);
    d.splits = reinterpret_cast<int4 *>(static_cast<uint8_t *>(ws) + sp.slots);
    d.whole = nullptr;
    d.ctas = kDecodeCtasPerSm * sm_count(dev);
    k.prefix = nullptr;
    k.splits = 0;
    int launches = 2;
    if (cache->prefix_len > 0) {
        d.whole = d.slots + (sp.slots + sp.list) / sizeof(float);
        k.splits = sp.splits;
        float *part = d.whole + sp.whole / sizeof(float);
        k.prefix = part;
        PagedTileArgs t = paged_tile_args(cache, a, sp.pairs, sp.splits, part);
        t.prefix_only = 1;
        if ((rc = cache->D == 64 ? launch_paged_tile_x<64>(cache, t, st)
                                 : launch_paged_tile_x<128>(cache, t, st)))
            return rc;
        ++launches;
    }
    const cudaError_t e = cache->D == 64 ? launch_paged_decode_x<64>(cache->dtype, k, st)
                                         : launch_paged_decode_x<128>(cache->dtype, k, st);
    if (e != cudaSuccess) return LWQ_ERR_CUDA;
    t_last_launches = launches;
    return LWQ_OK;
}

size_t lwq_attention_prefill_workspace_size(const lwq_paged *cache, int T, int H) {
    if (paged_sizes(cache, H) || T <= 0) return 0;
    int dev = 0, sms = 148;
    if (current_device(&dev) == LWQ_OK) sms = sm_count(dev);
    const size_t need = tile_part_most(tile_pairs(T, cache->B, H / cache->Hkv), cache->Hkv,
                                       (long)cache->max_pages * cache->page + cache->prefix_len, sms, cache->D, false);
    return need < 256 ? 256 : need;
}

int lwq_attention_prefill(const lwq_paged *cache, int flags, const void *q, void *out, const int32_t *cu_tokens,
                          int T, int H, float scale, void *stream) {
    t_last_launches = 0;
    PagedAttnArgs a;
    int rc = paged_attn_args(cache, flags, q, out, cu_tokens, T, H, scale, &a);
    if (rc) return rc;
    int dev;
    if ((rc = current_device(&dev))) return rc;
    long pairs;
    int splits;
    prefill_plan(cache, T, H, sm_count(dev), &pairs, &splits);
    if ((double)pairs * cache->Hkv * splits > (double)kMaxIndex) return LWQ_ERR_UNSUPPORTED;
    void *ws;
    if ((rc = paged_workspace(dev, splits > 1 ? tile_part_bytes(pairs, cache->Hkv, splits, cache->D) : 0, &ws))) return rc;
    PagedTileArgs t = paged_tile_args(cache, a, pairs, splits, static_cast<float *>(ws));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if ((rc = cache->D == 64 ? launch_paged_tile_x<64>(cache, t, st) : launch_paged_tile_x<128>(cache, t, st))) return rc;
    t_last_launches = splits > 1 ? 2 : 1;
    return LWQ_OK;
}

}  // extern "C"
