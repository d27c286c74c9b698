// The paged key/value cache: appending to it with the rotation of positions,
// and attention over it (see include/lwq.h, "paged key/value cache").
//
// Layout: pages [num_pages][Hkv][page][D], so that one page of one kv head is
// a contiguous run of page * D elements and a sequence's keys of a head are
// such runs, named by its row of the page table.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "../../include/lwq.h"
#include "lwq_attn.cuh"

namespace lwq {

// The cache as the kernels see it (lwq_paged with the derived sizes).
struct PagedArgs {
    uint16_t *k, *v;
    const int *tables, *lens, *prefix;
    int prefix_len;
    int B, Hkv, page, page_shift, max_pages, num_pages;
};

// The page that holds token j of a sequence (or of the prefix) with page list
// `list`, or -1 for a page number outside the cache (reported, never followed).
__device__ __forceinline__ int page_of(const PagedArgs &c, const int *list, int j) {
    const int p = __ldg(list + (j >> c.page_shift));
    if (p >= 0 && p < c.num_pages) return p;
    set_dev_error(DEVERR_BAD_PAGE);
    return -1;
}

// Element offset of token j's row within page p, kv head g.
template <int D>
__device__ __forceinline__ size_t cache_row(const PagedArgs &c, int p, int g, int j) {
    return (((size_t)p * c.Hkv + g) * c.page + (j & (c.page - 1))) * D;
}

// ------------------------------------------------------------------ append
// Rotation and append in one pass: every element of q, k and v is read once
// and written once, so the kernel is bound by HBM for long prompts and by the
// launch for single tokens.
//
// A group of D / 8 lanes takes one head of a token: 4 pairs per lane, i.e. 4 + 4
// (HALF) or 8 (PAIRS) consecutive elements, so that each warp-wide access is
// whole 128-byte lines; a warp takes 4 such accesses of one token's queries,
// keys or values with all their loads in flight before the first store, and no
// warp decides anything per head.  A block is one token's warps (up to 8: 40
// rotated and 8 other heads of 128 take 6), which share the (cos, sin) of the
// token's pairs: computed per warp they were half of all instructions (7776
// tokens, 48 heads of 128: 58.5 us, and 52 to 53 us shared: 5.4 TB/s).
//
// The angle position * f is kept in turns as a 64-bit fraction: the low 64 bits
// of position * turn are the exact product modulo one turn, and their top 32
// bits, as a signed fraction of a half turn, go to sincospi.  So a position of
// 2^31 costs no accuracy (fp32 angles would be off by whole turns there), and
// no 64-bit floating point is used.
constexpr int APPEND_ITERS = 4;
constexpr int APPEND_WARPS = 8;   // at most

struct AppendArgs {
    PagedArgs c;
    const void *q, *k, *v;
    long ldq, ldk, ldv;
    uint16_t *q_out;
    const int *cu, *positions;
    int T, H;
    int uq, uk;        // warps per token for q, and for k (and as many for v)
    int rope;          // 0: no rotation
    int pairs_layout;  // LWQ_ROPE_PAIRS
};

// 4 consecutive elements of a row in fp32 (ST: the source type).
template <int ST>
__device__ __forceinline__ void load4(const void *row, int e, float (&f)[4]) {
    if constexpr (ST == X_F32) {
        const float4 u = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(row) + e));
        f[0] = u.x;
        f[1] = u.y;
        f[2] = u.z;
        f[3] = u.w;
    } else {
        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(row) + e));
        f[0] = lo16<ST>(u.x);
        f[1] = hi16<ST>(u.x);
        f[2] = lo16<ST>(u.y);
        f[3] = hi16<ST>(u.y);
    }
}
template <int XT>
__device__ __forceinline__ void store4(uint16_t *p, const float (&f)[4]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack16<XT>(f[0], f[1]), pack16<XT>(f[2], f[3]));
}

template <int ST, int XT, int D>
__global__ void __launch_bounds__(APPEND_WARPS * 32) kv_append_kernel(const AppendArgs a, const lwq_rope rope) {
    constexpr int LPH = D / 8;          // lanes per head
    constexpr int HPI = 32 / LPH;       // heads per warp access
    __shared__ float2 trig[64];         // (cos, sin) of the token's pairs
    const int lane = threadIdx.x & 31, t = blockIdx.x;
    int unit = blockIdx.y * APPEND_WARPS + (threadIdx.x >> 5);
    const bool idle = unit >= a.uq + 2 * a.uk;   // (the last block of a token's)
    const PagedArgs &c = a.c;
    const int what = unit < a.uq ? 0 : unit < a.uq + a.uk ? 1 : 2;   // q, k, v
    unit -= what == 0 ? 0 : what == 1 ? a.uq : a.uq + a.uk;
    const int pi = lane % LPH, h0 = unit * APPEND_ITERS * HPI + lane / LPH, heads = what ? c.Hkv : a.H;
    const bool turned = a.rope && what < 2 && 8 * pi < rope.rot_dim;
    const bool halves = turned && !a.pairs_layout;
    // element offsets of the lane's two groups of four
    const int e0 = halves ? 4 * pi : 8 * pi;
    const int e1 = halves ? e0 + rope.rot_dim / 2 : e0 + 4;
    // the rows first: what follows looks up the token's place while they are on their way
    const long ld = what == 0 ? a.ldq : what == 1 ? a.ldk : a.ldv;
    const char *src = static_cast<const char *>(what == 0 ? a.q : what == 1 ? a.k : a.v) +
                      (t * ld + (long)h0 * D) * (ST == X_F32 ? 4 : 2);
    float x[APPEND_ITERS][2][4];
#pragma unroll
    for (int i = 0; i < APPEND_ITERS; ++i) {
        if (!idle && h0 + i * HPI < heads) {
            load4<ST>(src, e0 + i * HPI * D, x[i][0]);
            load4<ST>(src, e1 + i * HPI * D, x[i][1]);
        }
    }
    // the token's sequence b, its tokens' first row and count, and its length: a lane looks at one sequence, all three
    // words at once, so that only the page table's word waits for another
    int b = t, idx = 0, n = 1, len = 0;
    if (a.cu) {
        bool found = false;
        for (int i0 = 0; i0 < c.B && !found; i0 += 32) {
            const int i = min(i0 + lane, c.B - 1);
            const int lo = __ldg(a.cu + i), hi = __ldg(a.cu + i + 1), ln = __ldg(c.lens + i);
            const unsigned hit = __ballot_sync(0xffffffffu, t >= lo && t < hi);
            if (hit) {
                const int at = __ffs(hit) - 1;
                b = min(i0 + at, c.B - 1);
                idx = t - __shfl_sync(0xffffffffu, lo, at);
                n = __shfl_sync(0xffffffffu, hi - lo, at);
                len = __shfl_sync(0xffffffffu, ln, at);
                found = true;
            }
        }
        if (!found) return;             // behind the last sequence
    } else {
        len = __ldg(c.lens + b);
    }
    const long place = (long)len - n + idx;
    if (place < 0) return;              // padding
    if (a.rope) {
        if ((int)threadIdx.x < rope.rot_dim / 2) {
            const int p = a.positions ? __ldg(a.positions + (size_t)rope.axis[threadIdx.x] * a.T + t)
                                      : c.prefix_len + (int)place;
            const uint64_t turns = (uint64_t)(int64_t)p * rope.turn[threadIdx.x];
            const int half_turns = (int)(uint32_t)((turns + 0x80000000ull) >> 32);
            float sn, cs;
            sincospif((float)half_turns * 4.656612873077393e-10f, &sn, &cs);   // 2^-31
            trig[threadIdx.x] = make_float2(cs, sn);
        }
        __syncthreads();   // (the block is one token's: all of it left above, or none)
    }
    if (idle) return;
    float cs[4], sn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = turned ? trig[4 * pi + i] : make_float2(1.f, 0.f);
        cs[i] = v.x;
        sn[i] = v.y;
    }
    uint16_t *dst;
    size_t step = (size_t)HPI * D;      // from one of the warp's heads to its next
    if (what == 0) {
        dst = a.q_out + ((size_t)t * a.H + h0) * D;
    } else {
        int page = -1;
        if (place < (long)c.max_pages * c.page)
            page = page_of(c, c.tables + (size_t)b * c.max_pages, (int)place);
        else
            set_dev_error(DEVERR_BAD_PAGE);
        if (page < 0) return;
        dst = (what == 1 ? c.k : c.v) + cache_row<D>(c, page, h0, (int)place);
        step *= c.page;
    }
#pragma unroll
    for (int i = 0; i < APPEND_ITERS; ++i) {
        if (h0 + i * HPI >= heads) break;
        float(&u)[4] = x[i][0];
        float(&v)[4] = x[i][1];
        if (turned) {
            if (a.pairs_layout) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float p = u[2 * j], r = u[2 * j + 1];
                    u[2 * j] = p * cs[j] - r * sn[j];
                    u[2 * j + 1] = r * cs[j] + p * sn[j];
                    const float s = v[2 * j], z = v[2 * j + 1];
                    v[2 * j] = s * cs[j + 2] - z * sn[j + 2];
                    v[2 * j + 1] = z * cs[j + 2] + s * sn[j + 2];
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = u[j], r = v[j];
                    u[j] = p * cs[j] - r * sn[j];
                    v[j] = r * cs[j] + p * sn[j];
                }
            }
        }
        store4<XT>(dst + i * step + e0, u);
        store4<XT>(dst + i * step + e1, v);
    }
}

// --------------------------------------------------------------- attention
struct PagedAttnArgs {
    PagedArgs c;
    const uint16_t *q;
    void *out;
    const int *cu;      // null: one query per sequence
    int T, H, G;
    int out16;
    float qscale;       // scale * log2(e)
};

// floats of one partial result: m (log2 domain), l, two unused, acc[D]
__host__ __device__ constexpr int part_stride(int D) { return D + 4; }

// A list of `count` runs laid end to end, their lengths given by weight(i):
// all NT threads of a block build it together (each sums a stretch of runs) and
// then find the run that holds a place.  scratch: NT / 32 + 2 words of shared
// memory, free for other use after a barrier behind the last call.
template <int NT>
struct RunScan {
    int lo = 0, hi = 0;
    long excl = 0, mine = 0, all = 0;
    template <class W>
    __device__ __forceinline__ void build(int count, long *scratch, W weight) {
        const int per = (count + NT - 1) / NT, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        lo = min(count, (int)threadIdx.x * per);
        hi = min(count, lo + per);
        mine = 0;
        for (int i = lo; i < hi; ++i) mine += weight(i);
        long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) scratch[warp] = incl;
        __syncthreads();
        all = 0;
        excl = incl - mine;
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) {
            if (i < warp) excl += scratch[i];
            all += scratch[i];
        }
    }
    // The run that holds place `want` < all, and the sum of those before it.
    template <class W>
    __device__ __forceinline__ void locate(long want, long *scratch, int *run, long *before, W weight) const {
        if (want >= excl && want < excl + mine) {
            long at = excl;
            for (int i = lo; i < hi; ++i) {
                const long n = weight(i);
                if (want < at + n) {
                    scratch[NT / 32] = i;
                    scratch[NT / 32 + 1] = at;
                    break;
                }
                at += n;
            }
        }
        __syncthreads();
        *run = (int)scratch[NT / 32];
        *before = scratch[NT / 32 + 1];
    }
};

// The same by each warp for itself, 32 runs at a time, without a barrier: for
// short lists (a block-wide scan's barriers cost more than up to four rounds).
constexpr int WARP_RUNS = 128;
// false: place `want` lies behind the last run
template <class W>
__device__ __forceinline__ bool warp_run_locate(int count, long want, int *run, long *before, W weight) {
    const int lane = threadIdx.x & 31;
    long base = 0;
    for (int i0 = 0; i0 < count; i0 += 32) {
        const long mine = i0 + lane < count ? weight(i0 + lane) : 0;
        long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, want < base + incl);
        if (hit) {
            const int at = __ffs(hit) - 1;
            *run = i0 + at;
            *before = base + __shfl_sync(0xffffffffu, incl - mine, at);
            return true;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
}

}  // namespace lwq
