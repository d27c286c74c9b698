// Decode attention over the paged cache: one query token per sequence.
//
// Every key and value is read once per kv head, shared by its G = H / Hkv
// query heads, so HBM bounds the pass (2 x 2 x D bytes and 4 G D operations
// per key).  The keys of all (sequence, kv head) pairs are laid end to end as
// units of 64 keys, and the CTAs of one resident wave take equal runs of units:
// ragged lengths, a single long sequence and a large batch all fill the GPU,
// and the host needs to know none of the lengths.  A run may begin or end
// inside a pair; such a pair's partial results (running maximum, sum, weighted
// values) go to the workspace and a second kernel merges them, told by the CTA
// in whose run the pair begins how many there are.
//
// Within a CTA each of the 4 warps takes 16 of a unit's 64 keys (one page, as
// pages are at least 16 tokens) through its own cp.async ring, which runs
// ahead across units and pairs: the tensor cores form S = Q K^T and O += P V
// with mma.sync (m16n8k16), rows being the query heads.  The probabilities
// enter as sums of 16-bit parts: hi in MMA rows 0..7 and lo in rows 8..15 of
// one product; in bf16, whose two parts hold only 16 bits, a third part in a
// product of its own when the result is wanted in fp32.  fp16's parts end at
// 2^-24, whatever the probability, so they are taken of 2^15 p, the most that
// fp16 holds for p <= 1: 22 bits of every p above 2^-17 of a warp's largest, an
// error below 2^-40 of the largest for the others.  (Of p itself, the keys
// behind one that is e^16 above them lost up to half their weight.)
//
// Measured (32 query and 8 kv heads of 128): one sequence of 100003 tokens in 65
// us, 6.3 TB/s, and a merge of 7.5 us; 48 sequences of 0 to 8191 in 125 us, 6.6
// TB/s, and 4.5 us; one query head per kv head, 16 x 4096 tokens, in 166 us, 6.5
// TB/s.  A plain copy runs at 6.5 TB/s.
#pragma once

#include "lwq_paged.cuh"

namespace lwq {

constexpr int PD_WARPS = 4;
constexpr int PD_UNIT = 64;     // keys of a unit: 16 per warp

// 16 bytes from global to shared, or zeros (the source is not read then)
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool live) {
    const int n = live ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ int own_len(const PagedArgs &c, int b) {
    const int len = __ldg(c.lens + b), cap = c.max_pages * c.page;
    return len < 0 ? 0 : len > cap ? cap : len;
}
__device__ __forceinline__ int units_of(int len) { return (len + PD_UNIT - 1) / PD_UNIT; }

// The division of `total` units over n CTAs: the first r take q + 1, the others q (none, with fewer units than CTAs).
struct Runs {
    long q, r;
    __device__ __forceinline__ Runs(long total, int n) : q(total / n), r(total % n) {}
    __device__ __forceinline__ long start(int i) const { return q * i + (i < r ? i : r); }
    __device__ __forceinline__ int cta_of(long u) const {   // the CTA whose run holds unit u < total
        const long head = r * (q + 1);
        return (int)(u < head ? u / (q + 1) : r + (u - head) / q);
    }
};

struct PagedDecodeArgs {
    PagedAttnArgs a;
    float *slots;       // [ctas][2][G] partial results of a CTA's first and last pair
    int4 *splits;       // [ctas]: the pair (x: sequence, y: kv head) that begins in this run and ends in a later one;
                        // z: the CTAs that it spans (0: there is none), w: the first one's slot
    float *whole;       // [B][H] results of pairs that one CTA finished, when a prefix is still to be added; for any
                        // other pair, words 2 and 3 hold z and 2 * CTA + w of its entry above
    int ctas;
};

// A place in the list of units: pair (b, g), unit `u` of the pair's `n`.
struct UnitPos {
    int b, g, u, n, len;
};
__device__ __forceinline__ void next_unit(const PagedArgs &c, UnitPos &p) {
    if (++p.u < p.n) return;
    p.u = 0;
    if (++p.g < c.Hkv) return;
    p.g = 0;
    do {
        if (++p.b >= c.B) {
            p.n = 0;
            return;
        }
        p.len = own_len(c, p.b);
        p.n = units_of(p.len);
    } while (p.n == 0);
}

template <int D, int NG>
struct PagedDecodeSmem {
    // two CTAs per SM: 6 tiles of 16 keys in flight per warp at D = 64, 3 (2 beside the second head group) at 128
    static constexpr int STAGES = D == 64 ? (NG == 2 ? 4 : 6) : (NG == 2 ? 2 : 3);
    static constexpr uint32_t ROWB = 2 * D, TILEB = 16 * ROWB, STAGEB = 2 * TILEB;
    static constexpr size_t RING = (size_t)PD_WARPS * STAGES * STAGEB;
    // rows of the merge are 4 words apart in banks (8 heads at one bank each would make every store eight turns); two
    // CTAs of the largest form still fit an SM's 228 KB
    static constexpr int MROW = D + 4;
    static constexpr size_t MERGE = (size_t)PD_WARPS * 8 * NG * (MROW + 2) * 4;
    static constexpr size_t TOTAL = RING + MERGE + 64;   // and the scan's words
};

// NG: groups of 8 query heads (1 or 2); PARTS: 16-bit parts of a probability (2 or 3)
template <int XT, int D, int NG, int PARTS>
__global__ void __launch_bounds__(PD_WARPS * 32) paged_decode_kernel(const PagedDecodeArgs d) {
    using SM = PagedDecodeSmem<D, NG>;
    constexpr int ST = SM::STAGES, NCH = D / 8;
    constexpr float LIFT = XT == X_F16 ? 32768.f : 1.f;   // of the probabilities' parts, and so of o
    constexpr uint32_t ROWB = SM::ROWB, TILEB = SM::TILEB, STAGEB = SM::STAGEB;
    extern __shared__ __align__(128) uint8_t dsm[];
    // the scan's words, in the dynamic space (its limit is raised to all that a block may have)
    long *const scratch = reinterpret_cast<long *>(dsm + SM::RING + SM::MERGE);
    const PagedAttnArgs &a = d.a;
    const PagedArgs &c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t = lane & 3, G = a.G;

    // this CTA's run of units, and the sequence that it begins in
    auto units = [&](int b) { return units_of(own_len(c, b)); };
    RunScan<PD_WARPS * 32> scan;
    scan.build(c.B, scratch, units);
    const long total = scan.all * c.Hkv;
    const Runs runs(total, d.ctas);
    const long u0 = runs.start(blockIdx.x), u1 = runs.start(blockIdx.x + 1);
    if (threadIdx.x == 0) d.splits[blockIdx.x] = make_int4(0, 0, 0, 0);   // (this thread also writes the last word on it)
    // sequences with no token of their own: zeros, or nothing beside the prefix
    for (int b = blockIdx.x; b < c.B; b += d.ctas) {
        if (own_len(c, b) > 0) continue;
        for (int x = threadIdx.x; x < a.H * D; x += PD_WARPS * 32) {
            if (!d.whole) {
                if (a.out16)
                    static_cast<uint16_t *>(a.out)[(size_t)b * a.H * D + x] = 0;
                else
                    static_cast<float *>(a.out)[(size_t)b * a.H * D + x] = 0.f;
            } else if (x < a.H) {
                *reinterpret_cast<float4 *>(d.whole + ((size_t)b * a.H + x) * part_stride(D)) =
                    make_float4(-INFINITY, 0.f, 0.f, 0.f);
            }
        }
    }
    if (u0 >= u1) {
        pdl_wait();
        return;
    }
    UnitPos cur;
    long before;
    scan.locate(u0 / c.Hkv, scratch, &cur.b, &before, units);
    const int steps = (int)(u1 - u0);
    cur.len = own_len(c, cur.b);
    cur.n = units_of(cur.len);
    {
        const long rem = u0 - before * c.Hkv;
        cur.g = (int)(rem / cur.n);
        cur.u = (int)(rem % cur.n);
    }
    UnitPos ahead = cur;    // the unit whose keys are fetched next, and their page (looked up a unit ahead)
    auto lookup = [&](const UnitPos &p) {
        const int j = p.u * PD_UNIT + 16 * warp;
        return p.n > 0 && j < p.len ? __ldg(c.tables + (size_t)p.b * c.max_pages + (j >> c.page_shift)) : -1;
    };
    int page = lookup(ahead);
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(dsm) + (uint32_t)warp * ST * STAGEB;
    auto issue = [&](int i) {
        if (i < steps) {
            const int j0 = ahead.u * PD_UNIT + 16 * warp;
            if (j0 < ahead.len) {
                const bool ok = page >= 0 && page < c.num_pages;
                if (!ok && lane == 0) set_dev_error(DEVERR_BAD_PAGE);
                const size_t row0 = cache_row<D>(c, ok ? page : 0, ahead.g, j0);
                const uint32_t st = ring + (uint32_t)(i % ST) * STAGEB;
#pragma unroll
                for (int q = 0; q < 2 * 16 * NCH / 32; ++q) {
                    const int x = q * 32 + lane;
                    const int which = x / (16 * NCH), rem = x % (16 * NCH), r = rem / NCH, ch = rem % NCH;
                    const uint16_t *src = (which ? c.v : c.k) + row0 + (size_t)r * D + 8 * ch;
                    // rows past the last token hold anything: they come in as zeros
                    cp_async16_or_zero(st + which * TILEB + r * ROWB + ((ch ^ (r & 7)) << 4), src,
                                       ok && j0 + r < ahead.len);
                }
            }
            next_unit(c, ahead);
            page = lookup(ahead);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) issue(i);

    float(*sm_m)[8 * NG] = reinterpret_cast<float(*)[8 * NG]>(dsm + SM::RING);
    float(*sm_l)[8 * NG] = sm_m + PD_WARPS;
    float(*sm_o)[8 * NG][SM::MROW] =
        reinterpret_cast<float(*)[8 * NG][SM::MROW]>(dsm + SM::RING + 2 * PD_WARPS * 8 * NG * 4);

    uint32_t qa[D / 16][2 * NG];
    float o[NG][D / 8][4], m[NG], l[NG];
    // Q as the A operand: MMA row r is query head r of the kv head (rows >= G are zero)
    auto load_q = [&](const UnitPos &p) {
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) {
            const int h = 8 * gg + gr;
            const uint16_t *qr = a.q + ((size_t)p.b * a.H + (size_t)p.g * G + (h < G ? h : 0)) * D;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t x0 = __ldg(reinterpret_cast<const unsigned int *>(qr + 16 * ks + 2 * t));
                const uint32_t x1 = __ldg(reinterpret_cast<const unsigned int *>(qr + 16 * ks + 8 + 2 * t));
                qa[ks][2 * gg] = h < G ? x0 : 0u;
                qa[ks][2 * gg + 1] = h < G ? x1 : 0u;
            }
        }
    };
    auto clear = [&] {
#pragma unroll
        for (int gg = 0; gg < NG; ++gg) {
            m[gg] = -INFINITY;
            l[gg] = 0.f;
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[gg][n][e] = 0.f;
        }
    };
    load_q(cur);
    clear();
    int pair = 0;   // pairs of this run so far
    for (int i = 0; i < steps; ++i) {
        issue(i + ST - 1);
        cp_async_wait<ST - 1>();
        __syncwarp();   // every lane's copies of step i are in and visible to the warp
        const uint32_t st = ring + (uint32_t)(i % ST) * STAGEB;
        const int j0 = cur.u * PD_UNIT + 16 * warp;
        if (j0 < cur.len) {
            float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            {
                const int key = (lane & 7) + ((lane >> 4) << 3), hcol = (lane >> 3) & 1;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    uint32_t r[4];
                    ldsm_x4(st + key * ROWB + (((2 * ks + hcol) ^ (key & 7)) << 4), r);
                    const uint32_t aq[4] = {qa[ks][0], NG == 2 ? qa[ks][2 * NG - 2] : 0u, qa[ks][1],
                                            NG == 2 ? qa[ks][2 * NG - 1] : 0u};
                    if constexpr (XT == X_F16) {
                        mma_f16_16816(sc[0], aq, r[0], r[1], sc[0]);
                        mma_f16_16816(sc[1], aq, r[2], r[3], sc[1]);
                    } else {
                        mma_bf16_16816(sc[0], aq, r[0], r[1], sc[0]);
                        mma_bf16_16816(sc[1], aq, r[2], r[3], sc[1]);
                    }
                }
            }
            uint32_t ap[NG][4], ap3[NG][4];
            float corr[NG];
#pragma unroll
            for (int gg = 0; gg < NG; ++gg) {
                // head 8 gg + gr's scores of keys 2t, 2t + 1, 8 + 2t, 9 + 2t, in the log2 domain
                float p[4] = {sc[0][2 * gg], sc[0][2 * gg + 1], sc[1][2 * gg], sc[1][2 * gg + 1]};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = 8 * (e >> 1) + 2 * t + (e & 1);
                    p[e] = j0 + key < cur.len ? p[e] * a.qscale : -INFINITY;
                }
                float mx = fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = fmaxf(m[gg], mx), base = mn == -INFINITY ? 0.f : mn;   // (scores may be -inf)
                corr[gg] = exp2f(m[gg] - base);         // 0 on the first step (m = -inf)
                float ps = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[e] = exp2f(p[e] - base);          // 0 for a key past the end
                    ps += p[e];
                }
                l[gg] = fmaf(l[gg], corr[gg], ps);
                m[gg] = mn;
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] *= LIFT;
                const uint32_t h0 = pack16<XT>(p[0], p[1]), h1 = pack16<XT>(p[2], p[3]);
                const float r0 = p[0] - lo16<XT>(h0), r1 = p[1] - hi16<XT>(h0);
                const float r2 = p[2] - lo16<XT>(h1), r3 = p[3] - hi16<XT>(h1);
                const uint32_t l0 = pack16<XT>(r0, r1), l1 = pack16<XT>(r2, r3);
                ap[gg][0] = h0;
                ap[gg][1] = l0;
                ap[gg][2] = h1;
                ap[gg][3] = l1;
                if constexpr (PARTS == 3) {
                    ap3[gg][0] = pack16<XT>(r0 - lo16<XT>(l0), r1 - hi16<XT>(l0));
                    ap3[gg][1] = 0u;
                    ap3[gg][2] = pack16<XT>(r2 - lo16<XT>(l1), r3 - hi16<XT>(l1));
                    ap3[gg][3] = 0u;
                }
            }
            const int key = (lane & 7) + (((lane >> 3) & 1) << 3), hcol = lane >> 4;
#pragma unroll
            for (int p2 = 0; p2 < D / 16; ++p2) {
                uint32_t r[4];
                ldsm_x4_t(st + TILEB + key * ROWB + (((2 * p2 + hcol) ^ (key & 7)) << 4), r);
#pragma unroll
                for (int gg = 0; gg < NG; ++gg) {
                    // the products of these 16 keys alone: the tensor cores truncate what they add up, which over
                    // many steps would pull every sum towards zero (1.2e-6 of the result after 64 steps, against
                    // 3e-7 this way), so the running sum is kept here, rescaled and added in one rounded FMA
                    float x0[4] = {0.f, 0.f, 0.f, 0.f}, x1[4] = {0.f, 0.f, 0.f, 0.f};
                    if constexpr (XT == X_F16) {
                        mma_f16_16816(x0, ap[gg], r[0], r[1], x0);
                        mma_f16_16816(x1, ap[gg], r[2], r[3], x1);
                    } else {
                        if constexpr (PARTS == 3) {
                            mma_bf16_16816(x0, ap3[gg], r[0], r[1], x0);
                            mma_bf16_16816(x1, ap3[gg], r[2], r[3], x1);
                        }
                        mma_bf16_16816(x0, ap[gg], r[0], r[1], x0);
                        mma_bf16_16816(x1, ap[gg], r[2], r[3], x1);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        o[gg][2 * p2][e] = fmaf(o[gg][2 * p2][e], corr[gg], x0[e]);
                        o[gg][2 * p2 + 1][e] = fmaf(o[gg][2 * p2 + 1][e], corr[gg], x1[e]);
                    }
                }
            }
        }
        __syncwarp();   // the stage is read before a later step's copies refill it

        const bool end_of_pair = cur.u + 1 == cur.n, last = i + 1 == steps;
        UnitPos next = cur;
        next_unit(c, next);
        if (end_of_pair || last) {
            if (!last) load_q(next);   // the next pair's queries arrive under the merge
            // merge the warps: per head the largest running maximum, the others rescaled to it
#pragma unroll
            for (int gg = 0; gg < NG; ++gg) {
                const int h = 8 * gg + gr;
                float ls = l[gg];
                ls += __shfl_xor_sync(0xffffffffu, ls, 1);
                ls += __shfl_xor_sync(0xffffffffu, ls, 2);
                if (t == 0) {
                    sm_m[warp][h] = m[gg];
                    sm_l[warp][h] = ls;
                }
#pragma unroll
                for (int n = 0; n < D / 8; ++n)   // hi rows + lo rows
                    if (h < G)
                        *reinterpret_cast<float2 *>(&sm_o[warp][h][8 * n + 2 * t]) =
                            make_float2((o[gg][n][0] + o[gg][n][2]) * (1.f / LIFT),
                                        (o[gg][n][1] + o[gg][n][3]) * (1.f / LIFT));
            }
            __syncthreads();
            // a pair that this run began and finished is complete; any other is a part of one
            const bool complete = end_of_pair && (pair > 0 || i + 1 >= cur.n);
            for (int x = threadIdx.x; x < G * D; x += PD_WARPS * 32) {
                const int h = x / D, e = x % D;
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < PD_WARPS; ++w) M = fmaxf(M, sm_m[w][h]);
                const float base = M == -INFINITY ? 0.f : M;
                float L = 0.f, A = 0.f;
#pragma unroll
                for (int w = 0; w < PD_WARPS; ++w) {
                    const float f = exp2f(sm_m[w][h] - base);
                    L = fmaf(sm_l[w][h], f, L);
                    A = fmaf(sm_o[w][h][e], f, A);
                }
                const size_t bh = (size_t)cur.b * a.H + (size_t)cur.g * G + h;
                if (complete && !d.whole) {
                    if (a.out16)
                        static_cast<uint16_t *>(a.out)[bh * D + e] = (uint16_t)pack16<XT>(A / L, 0.f);
                    else
                        static_cast<float *>(a.out)[bh * D + e] = A / L;
                } else {
                    float *pp = complete ? d.whole + bh * part_stride(D)
                                         : d.slots + (((size_t)blockIdx.x * 2 + (pair > 0)) * G + h) * part_stride(D);
                    if (e == 0) *reinterpret_cast<float4 *>(pp) = make_float4(M, L, 0.f, 0.f);
                    pp[4 + e] = A;
                }
            }
            if (!end_of_pair && (pair > 0 || i + 1 == cur.u + 1)) {
                // the pair begins in this run (`i + 1 == cur.u + 1`: with its first unit) and goes on in later ones
                const long end = u1 + (cur.n - 1 - cur.u);   // past its last unit
                const int count = runs.cta_of(end - 1) - (int)blockIdx.x + 1, slot = pair > 0;
                if (threadIdx.x == 0) d.splits[blockIdx.x] = make_int4(cur.b, cur.g, count, slot);
                if (d.whole && threadIdx.x < G)
                    *reinterpret_cast<float4 *>(d.whole + ((size_t)cur.b * a.H + (size_t)cur.g * G + threadIdx.x) *
                                                              part_stride(D)) =
                        make_float4(0.f, 0.f, __int_as_float(count), __int_as_float(2 * blockIdx.x + slot));
            }
            __syncthreads();   // the merge space is free again
            ++pair;
            clear();
        }
        cur = next;
    }
    pdl_launch_dependents();
    pdl_wait();   // a prefix's row tiles, which this kernel does not read, end before it does
}

// One step of a merge: a partial result (m, l, one value) joins (M, L, A).
template <int E>
__device__ __forceinline__ void merge_part(float &M, float &L, float (&A)[E], float m, float l, const float (&v)[E]) {
    if (m == -INFINITY) return;
    const float mn = fmaxf(M, m), fo = exp2f(M - mn), fn = exp2f(m - mn);   // fo = 0 while M = -inf
    L = fmaf(L, fo, l * fn);
#pragma unroll
    for (int e = 0; e < E; ++e) A[e] = fmaf(A[e], fo, v[e] * fn);
    M = mn;
}
template <int XT>
__device__ __forceinline__ void store_out(const PagedAttnArgs &a, size_t at, float v) {
    if (a.out16)
        static_cast<uint16_t *>(a.out)[at] = (uint16_t)pack16<XT>(v, 0.f);
    else
        static_cast<float *>(a.out)[at] = v;
}

// Merges the pairs that several CTAs worked on.  `parts` blocks per CTA in whose
// run such a pair begins (most have none) share its G * D columns; a block's
// threads take its columns in as many groups as fit, each group every so-manieth
// partial result, eight loads in flight.  The order of every addition is fixed
// by the sizes.  One block per CTA does for pairs cut in two or three (4.0 us
// after the 125 us of 48 ragged sequences; a block per head 6.4 us, most of it
// blocks that find nothing to do); a pair over 37 CTAs wants a block per head
// (one sequence of 100003 tokens: 7 us, against 12 us).
constexpr int PC_THREADS = 512;
inline int combine_parts(long pairs, int G, int ctas) { return 4 * pairs <= ctas ? G : 1; }
template <int XT, int D>
__global__ void __launch_bounds__(PC_THREADS) paged_combine_kernel(const PagedDecodeArgs d, int parts) {
    constexpr int PS = part_stride(D), U = 8;
    __shared__ float gm[PC_THREADS], gl[PC_THREADS], go[PC_THREADS];
    const PagedAttnArgs &a = d.a;
    const int i0 = blockIdx.x / parts, n = a.G * D / parts, c0 = (blockIdx.x % parts) * n;   // columns [c0, c0 + n)
    pdl_wait();
    const int4 sp = __ldcg(d.splits + i0);
    if (sp.z == 0) return;
    const int groups = n < (int)blockDim.x ? (int)blockDim.x / n : 1, grp = groups > 1 ? threadIdx.x / n : 0;
    for (int x = groups > 1 ? threadIdx.x % n : threadIdx.x; x < n; x += blockDim.x) {
        const int col = c0 + x, h = col / D, e = col % D;
        float M = -INFINITY, L = 0.f, A[1] = {0.f};
        for (int s0 = grp; s0 < sp.z; s0 += groups * U) {
            float mv[U], lv[U], av[U][1];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int s = s0 + u * groups < sp.z ? s0 + u * groups : 0;
                const float *p = d.slots + (((size_t)(i0 + s) * 2 + (s == 0 ? sp.w : 0)) * a.G + h) * PS;
                const float2 ml = __ldcg(reinterpret_cast<const float2 *>(p));
                mv[u] = s0 + u * groups < sp.z ? ml.x : -INFINITY;
                lv[u] = ml.y;
                av[u][0] = __ldcg(p + 4 + e);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) merge_part(M, L, A, mv[u], lv[u], av[u]);
        }
        if (groups > 1) {   // (blockDim.x is then a multiple of n: one round, every thread takes part)
            gm[threadIdx.x] = M;
            gl[threadIdx.x] = L;
            go[threadIdx.x] = A[0];
            __syncthreads();
            if (grp > 0) return;
            for (int i = 1; i < groups; ++i) {
                const float v[1] = {go[i * n + x]};
                merge_part(M, L, A, gm[i * n + x], gl[i * n + x], v);
            }
        }
        store_out<XT>(a, ((size_t)sp.x * a.H + (size_t)sp.y * a.G) * D + col, A[0] / L);
    }
}

// Adds the prefix's partial results to each row's own: a warp per (sequence,
// query head), its lanes the columns.
struct PagedPrefixArgs {
    PagedDecodeArgs d;
    const float *prefix;     // [(row / 256 * Hkv + g) * splits + s][256] rows, row = b G + h
    int splits;
};
template <int XT, int D>
__global__ void __launch_bounds__(256) paged_prefix_combine_kernel(const PagedPrefixArgs k) {
    constexpr int E = D / 32, PS = part_stride(D), U = 4;
    const PagedAttnArgs &a = k.d.a;
    const long w = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    pdl_wait();
    if (w >= (long)a.c.B * a.H) return;
    const int b = (int)(w / a.H), hh = (int)(w % a.H), g = hh / a.G, h = hh % a.G;
    const long row = (long)b * a.G + h;
    const float *pre = k.prefix + ((((row >> 8) * a.c.Hkv + g) * k.splits) * 256 + (row & 255)) * PS;
    const float *own = k.d.whole + (size_t)w * PS;
    const float4 head = __ldcg(reinterpret_cast<const float4 *>(own));
    const int count = __float_as_int(head.z), first = __float_as_int(head.w);
    float M = -INFINITY, L = 0.f, A[E];
#pragma unroll
    for (int e = 0; e < E; ++e) A[e] = 0.f;
    const int total = k.splits + (count ? count : 1);
    for (int s0 = 0; s0 < total; s0 += U) {
        float mv[U], lv[U], av[U][E];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + u, o = s - k.splits;
            const float *p = pre;
            if (s < k.splits)
                p = pre + (size_t)s * 256 * PS;
            else if (s < total)
                p = count == 0 ? own : k.d.slots + (((size_t)(first / 2 + o) * 2 + (o == 0 ? first & 1 : 0)) * a.G + h) * PS;
            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(p));
            mv[u] = s < total ? ml.x : -INFINITY;
            lv[u] = ml.y;
#pragma unroll
            for (int e = 0; e < E; ++e) av[u][e] = __ldcg(p + 4 + 32 * e + lane);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) merge_part(M, L, A, mv[u], lv[u], av[u]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) store_out<XT>(a, (size_t)w * D + 32 * e + lane, A[e] / L);   // the prefix has a token
}

}  // namespace lwq
