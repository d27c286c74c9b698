// Attention of many query rows over one run of keys, on the tcgen05 tensor
// cores: the prefill of a sequence's new tokens (causal), and a shared prefix
// against the queries of a whole batch.
//
// Rows are (token, query head) pairs of one kv head, row = token * G + head, so
// that every G fills the 128 rows of an MMA and a key tile is read once for all
// the heads that share it.  A CTA takes 256 rows (two MMA tiles) of one
// sequence and kv head, and a contiguous part of the key tiles (all of them
// when there are enough rows to fill the GPU; partial results are merged by a
// second kernel otherwise):
//
//   warp 0      TMA: key and value tiles through one ring, K0 V0 K1 V1 ...;
//               a tile is as many boxes as pages it spans
//   warp 1      tcgen05.mma: S_t = Q_t K^T (both from shared memory), then
//               O_t += P_t V with P_t in TMEM, over S_t's columns
//   warp 2      answers for tiles that have landed, and clears the value rows
//               behind a segment's last key (warp 3 idles)
//   warps 4..11 softmax, one thread per row: S_t from TMEM, running maximum
//               and sum in fp32, P_t back to TMEM
//
// The two row tiles alternate: while one's scores are in the softmax warps the
// tensor core works on the other.  A row's output is rescaled only when its
// running maximum has outgrown the one that its probabilities are taken
// against (see TileRange): until then they are larger by a factor, in numerator
// and denominator alike.
//
// The probabilities are PARTS 16-bit numbers each.  A 16-bit result takes one
// part (off by half a step of that type per key, like the result's own
// rounding); an fp32 result takes two in fp16 (22 bits; fp16's parts end at
// 2^-24, whatever the probability, so they are taken of 2^10 to 2^15 p), three
// in bf16 (24).
// The tensor cores truncate what they add to O, which pulls every sum towards
// zero by about 2^-23 per product of 16 keys; for an fp32 result O therefore
// starts anew every 1024 keys and the sums so far are kept, in rounded fp32,
// in the row's place in the output (or among the partial results): at any length
// 2e-6 (bf16) and 7e-6 (fp16) of a result whose values have one sign, 1 to 2e-6
// of sum p |v| otherwise.  For a 16-bit result it is relieved every 16384 keys
// in fp16, every 32768 in bf16 (1e-4 and 2e-4 of the result, a fifth and a
// twentieth of a half step; 131072 keys left to one accumulator took 8e-4, nearly
// two half steps of fp16): the row's place in the output takes the sums so far
// rounded to 16 bits, in units of a power of two that holds them, and O goes on
// from the remainder, so that nothing is lost and no fp32 space is needed.  Each
// time costs a CTA about 10 us (16384 tokens relieved every 8192 keys took 2.10
// ms, never 2.01), so it is not done more often.
//
// Measured (32 query and 8 kv heads of 128, bf16, other inputs each time): a
// prompt of 8192 tokens in 515 to 535 us, 1.03 to 1.07 PFLOP/s, 0.61 to 0.64 of
// what a large matrix product reaches in a burst (0.74 to 0.77 of what it
// sustains); 16384 tokens in 1.94 ms, 1.13 PFLOP/s; 8192 with an fp32 result in
// 1.06 ms, fp16 0.93.  A key tile of both row tiles takes about 3000 cycles, of
// which the tensor core works 2050: one row tile's softmax (2000 cycles) and the
// products behind it (900) form a chain, and 7 us of a CTA's life are its start
// and end.
#pragma once

#include "lwq_paged_decode.cuh"

namespace lwq {

constexpr int TILE_ROWS = 128;
constexpr int PAIR_ROWS = 2 * TILE_ROWS;
constexpr int TILE_THREADS = 384;
// registers per thread after the split: 128 x 56 + 256 x 224 = 64512, the 384 x 168 of the launch
constexpr int TILE_REGS_FEED = 56, TILE_REGS_SOFTMAX = 224;
constexpr uint32_t TILE_TMEM_COLS = 512;
// What a row's probabilities are taken against (m, in the log2 domain, as all exponents here): when its maximum `top` is
// taken anew they begin at 2^LIFT, and until one would pass 2^ROOM a larger score changes nothing.
//   bf16   has fp32's range: 0 and 8.
//   fp16   ends at 2^-24 below and at 65504 above: ROOM is 15, the half that stays free being for the rounding of
//          exponents up to EXACT in size.  Begun at 2^10, a row's weights are off by less than 2^-35 of its largest.
//          Higher up they outgrow the room too often (fp32 results: at 2^11 ragged prompts take 80 to 84 us instead of
//          76.6, at 2^13 a prompt of 8192 tokens 1105 instead of 930).  But a key that stands alone above the tile's
//          others by more than ALONE (an attention sink: nothing follows that comes near it) begins at 2^15, and they
//          are off by 2^-40 of it: there the others' weights may be all that the result is made of, while without such
//          a key weights within 2^-8 of the largest outweigh what is lost.  Beyond EXACT, where 15 would be lost in the
//          rounding of the maximum itself, 0 and 2: scores of up to 2^27, off by up to 8 from their maximum, stay in
//          the type.
template <int XT>
struct TileRange {
    static constexpr float LIFT = XT == X_F16 ? 10.f : 0.f, ROOM = XT == X_F16 ? 15.f : 8.f;
    static constexpr float ALONE = 8.f, ALONE_LIFT = 15.f, EXACT = 4194304.f, FAR_ROOM = 2.f;
};

struct PagedTileArgs {
    PagedAttnArgs a;
    float *part;        // partial results [(pair * Hkv + g) * splits + s][256 rows], or null: write out
    int splits;
    long pairs;         // of row tiles that the call has room for
    int prefix_only;    // the batch's queries (one row set of all T tokens) against the prefix alone
    int flip;           // negative scale: Q's signs are flipped and qscale is positive
    int total_rows;     // cache rows (num_pages Hkv page): the coordinate of a page that is not there
    unsigned long long timeout_ns;
};

// pairs of row tiles of a sequence with n new tokens
__host__ __device__ __forceinline__ long pairs_of(long n, int G) { return n <= 0 ? 0 : (n * G + PAIR_ROWS - 1) / PAIR_ROWS; }

// The tokens of sequence b: its first row of q, and how many (none where cu does not ascend, none past T).
__device__ __forceinline__ int first_token(const PagedAttnArgs &a, int b) {
    return a.cu ? min(max(__ldg(a.cu + b), 0), a.T) : b;
}
__device__ __forceinline__ int token_count(const PagedAttnArgs &a, int b) {
    return a.cu ? max(min(__ldg(a.cu + b + 1), a.T) - first_token(a, b), 0) : 1;
}

// The rows of one pair: its sequence, first row, and what its rows see.
struct RowSet {
    int b, tok0, n;     // sequence, its first token's row of q, its tokens
    int row0;           // first row of the pair among the sequence's n * G
    int len;            // the sequence's tokens in the cache, at most what its page table holds
};
// tokens seen before and at row r: -1 for a row that sees nothing, else the sequence's own tokens
__device__ __forceinline__ int own_seen(const RowSet &s, int G, int r) {
    const long place = (long)s.len - s.n + r / G;
    return place < 0 ? -1 : (int)(place + 1);
}

template <int D, int KT>
struct TileSmem {
    static constexpr uint32_t HALVES = D / 64;                       // 64-element (128-byte) column groups
    static constexpr uint32_t HALF_Q = TILE_ROWS * 128, HALF_KV = KT * 128;
    static constexpr uint32_t QB = HALVES * HALF_Q, SLOT = HALVES * HALF_KV;
    static constexpr int STAGES = (227 * 1024 - 2 * QB - 2048) / SLOT < 8 ? (227 * 1024 - 2 * QB - 2048) / SLOT : 8;
    static constexpr size_t BARS = 2 * QB + STAGES * SLOT;           // offset of the barriers
    static constexpr size_t TOTAL = 1024 + BARS + 256;
};

__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Operand whose rows are contiguous along N (values [key][D]): 64-element column groups `lead` bytes apart, 8-key
// groups 1024 bytes apart, 128-byte swizzle.
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t smem_addr, uint32_t lead) {
    return (uint64_t)((smem_addr & 0x3FFFFu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A warpgroup's registers per thread (all of its warps take part).
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Pairs of fp32 values in one 64-bit register, and the packed instructions on them.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

template <int XT, int D, int PARTS, int KT>
__global__ void __launch_bounds__(TILE_THREADS, 1)
    paged_tile_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                      const PagedTileArgs ta) {
    using SM = TileSmem<D, KT>;
    static_assert(PARTS * KT / 2 <= 128 && KT <= 128 && KT % 64 == 0, "a tile's scores and probabilities share 128 columns");
    static_assert(SM::STAGES >= 4, "V and the next K land before a tile's products, which hand back the V before them");
    constexpr int ST = SM::STAGES;
    constexpr int FRESH = PARTS > 1 ? 1024 / KT : 1 << 30;   // key tiles after which O starts anew
    constexpr int RELIEF = (XT == X_F16 ? 16384 : 32768) / KT;   // with one part: after which it goes on from a remainder
    constexpr int SPLIT = KT == 128 ? 96 : 32;   // keys of the first part of the probabilities
    constexpr uint32_t IDESC_S = umma_idesc_f16(XT == X_F16 ? 0 : 1, TILE_ROWS, KT);
    constexpr uint32_t IDESC_O = umma_idesc_f16(XT == X_F16 ? 0 : 1, TILE_ROWS, D) | (1u << 16);   // B along N
    extern __shared__ uint8_t raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const PagedAttnArgs &a = ta.a;
    const PagedArgs &c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + SM::BARS);
    uint64_t *full = bars, *empty = bars + ST, *q_full = bars + 2 * ST, *s_full = q_full + 2, *p_full = s_full + 2,
             *o_full = p_full + 4, *all_done = o_full + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(all_done + 1);

    // ---- which rows, which kv head, which part of the keys
    const int group = c.Hkv * ta.splits;
    const int g = (int)(blockIdx.x % group) / ta.splits, split = (int)(blockIdx.x % ta.splits);
    const long pair = blockIdx.x / group;
    RowSet rs;
    long pl;
    if (ta.prefix_only) {
        rs.b = 0;
        rs.tok0 = 0;
        rs.n = a.T;
        rs.len = 0;
        pl = pair;
    } else {
        auto weight = [&](int b) { return pairs_of(token_count(a, b), a.G); };
        long before;
        if (threadIdx.x < c.B) asm volatile("prefetch.global.L1 [%0];" ::"l"(c.lens + threadIdx.x));
        if (c.B <= WARP_RUNS) {
            if (!warp_run_locate(c.B, pair, &rs.b, &before, weight)) return;
        } else {
            long *scratch = reinterpret_cast<long *>(sm);
            RunScan<TILE_THREADS> scan;
            scan.build(c.B, scratch, weight);
            if (pair >= scan.all) return;
            scan.locate(pair, scratch, &rs.b, &before, weight);
            __syncthreads();   // the scratch is shared memory of the tiles
        }
        rs.tok0 = first_token(a, rs.b);
        rs.n = token_count(a, rs.b);
        rs.len = min(__ldg(c.lens + rs.b), c.max_pages * c.page);
        pl = pairs_of(rs.n, a.G) - 1 - (pair - before);   // the rows that see most first
    }
    rs.row0 = (int)(pl * PAIR_ROWS);
    const int rows = min(rs.n * a.G - rs.row0, PAIR_ROWS);   // live rows of the pair
    const int npre = (c.prefix_len + KT - 1) / KT;
    // key tiles that row tile t sees, and those of the pair; this CTA takes [j0, j1) of the latter
    auto tiles_seen = [&](int t) {
        const int live = min(rows - t * TILE_ROWS, TILE_ROWS);
        if (live <= 0) return 0;
        if (ta.prefix_only) return npre;
        const int seen = own_seen(rs, a.G, rs.row0 + t * TILE_ROWS + live - 1);
        return seen < 0 ? 0 : npre + (seen + KT - 1) / KT;
    };
    const int n0 = tiles_seen(0), n1 = tiles_seen(1), nall = max(n0, n1);
    const int own_load = ta.prefix_only ? 0 : max(0, own_seen(rs, a.G, rs.row0 + rows - 1));
    const int j0 = (int)((long)nall * split / ta.splits), j1 = (int)((long)nall * (split + 1) / ta.splits);
    const int cnt0 = min(max(n0 - j0, 0), j1 - j0), cnt1 = min(max(n1 - j0, 0), j1 - j0), cnt = max(cnt0, cnt1);

    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&q_full[t], 4);
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[t], 5);       // four softmax warps, and warp 2
            mbar_init(&p_full[t + 2], 4);
            mbar_init(&o_full[t], 1);
        }
        mbar_init(all_done, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, TILE_TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = *tmem_holder;
    auto s_col = [&](int t) { return tmem + 128u * t; };
    auto o_col = [&](int t) { return tmem + 256u + 128u * t; };
    const uint32_t q_smem = smem_u32(sm), ring = q_smem + 2 * SM::QB;
    // key tile j of the pair: its first key within its segment, and its live keys
    auto tile_keys = [&](int j, int *key0) {
        if (j < npre) {
            *key0 = j * KT;
            return min(KT, c.prefix_len - j * KT);
        }
        *key0 = (j - npre) * KT;
        return min(KT, own_load - *key0);
    };

    // a warp's wait, by one of its lanes
    auto warp_wait = [&](uint64_t *bar, uint32_t parity) {
        int ok = 1;
        if (lane == 0) ok = mbar_wait_near(bar, parity, ta.timeout_ns, DEVERR_ATTN_WAIT);
        return __shfl_sync(0xffffffffu, ok, 0) != 0;
    };
    // one by all of its lanes, each on its own, as a chain of short steps wants it; they agree on how it ended, since what
    // follows takes the whole warp (near the limit some could give up and others not)
    auto all_wait = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait_near(bar, parity, ta.timeout_ns, DEVERR_ATTN_WAIT)) != 0;
    };
    // (the register split is one instruction for all of a warpgroup's warps)
    if (warp < 4) {
        regs_dec<TILE_REGS_FEED>();
        if (warp == 0) {
            // -------------------------------------------------------------- TMA
            const int brows = min(c.page, KT);
            const int *table = c.tables + (size_t)rs.b * c.max_pages;
            bool ok = true;
            int i = 0;
            for (int j = j0; ok && j < j0 + cnt; ++j) {
                int key0;
                const int valid = tile_keys(j, &key0);
                const int boxes = (valid + brows - 1) / brows;
                const int box = lane / (int)SM::HALVES, half = lane % (int)SM::HALVES;
                int row = 0;
                if (box < boxes) {
                    const int p = page_of(c, j < npre ? c.prefix : table, key0 + box * brows);
                    row = p < 0 ? ta.total_rows : (p * c.Hkv + g) * c.page + ((key0 + box * brows) & (c.page - 1));
                }
                for (int w = 0; w < 2; ++w, ++i) {
                    const int slot = i % ST;
                    if (i >= ST && !(ok = warp_wait(&empty[slot], (uint32_t)((i / ST - 1) & 1))))
                        break;
                    if (lane == 0) mbar_arrive_expect_tx(&full[slot], (uint32_t)(boxes * brows * D * 2));
                    __syncwarp();
                    if (box < boxes)
                        tma_load_2d(sm + 2 * SM::QB + (size_t)slot * SM::SLOT + half * SM::HALF_KV + (size_t)box * brows * 128,
                                    w ? &vmap : &kmap, &full[slot], half * 64, row);
                }
            }
            // copies still in flight land before the block ends
            for (int x = max(0, i - ST); x < i; ++x)
                warp_wait(&full[x % ST], (uint32_t)((x / ST) & 1));
        } else if (warp == 1) {
            // -------------------------------------------------------------- MMA
            // One thread.  What lies between the arrival of probabilities and the next products is the critical path, so
            // it waits for nothing else (warp 2 answers for the tiles in shared memory, as one of the arrivals on the
            // probabilities' barrier); descriptors are made once and advanced by adding, and a tile's slots are handed
            // back late, behind the next tile's first products (a commit is not issued before the products ahead of it).
            if (elect_one()) {
                bool ok = true;
                int slot = 0;           // of the ring
                const uint64_t q_desc = umma_desc_sw128(q_smem), k_desc = umma_desc_sw128(ring),
                               v_desc = umma_desc_mn_sw128(ring, SM::HALF_KV);
                auto scores = [&](int t, int at) {   // S_t = Q_t K^T, the keys in slot `at`
                    const uint64_t qd = q_desc + (uint64_t)(t * (SM::QB >> 4)), kd = k_desc + (uint64_t)(at * (SM::SLOT >> 4));
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        umma_f16(s_col(t), qd + ((kk / 4) * SM::HALF_Q + (kk % 4) * 32) / 16,
                                 kd + ((kk / 4) * SM::HALF_KV + (kk % 4) * 32) / 16, IDESC_S, kk ? 1u : 0u);
                    umma_commit(&s_full[t]);
                };
                int back[2] = {-1, -1};   // slots to hand back
                if (cnt > 0) {
                    ok = mbar_wait_near(&full[0], 0, ta.timeout_ns, DEVERR_ATTN_WAIT);
                    for (int t = 0; ok && t < 2; ++t) {
                        if ((t ? cnt1 : cnt0) == 0) continue;
                        if (!(ok = mbar_wait_near(&q_full[t], 0, ta.timeout_ns, DEVERR_ATTN_WAIT))) break;
                        scores(t, 0);
                    }
                    back[0] = 0;
                    for (int j = 0; ok && j < cnt; ++j) {
                        const int v_slot = slot + 1 < ST ? slot + 1 : 0, k_slot = v_slot + 1 < ST ? v_slot + 1 : 0;
                        slot = k_slot;
                        const uint64_t vd = v_desc + (uint64_t)(v_slot * (SM::SLOT >> 4));
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const int mine = t ? cnt1 : cnt0;
                            if (!ok || j >= mine) continue;
                            // the probabilities come in two parts, so that the products of the first overlap the
                            // exponentials of the second
#pragma unroll
                            for (int part = 0; part < 2; ++part) {
                                if (ok) ok = mbar_wait_near(&p_full[t + 2 * part], (uint32_t)(j & 1), ta.timeout_ns, DEVERR_ATTN_WAIT);
                                if (!ok) continue;
                                tc_fence_after();
#pragma unroll
                                for (int p = PARTS - 1; p >= 0; --p)
#pragma unroll
                                    for (int kk = part ? SPLIT / 16 : 0; kk < (part ? KT / 16 : SPLIT / 16); ++kk)
                                        umma_f16_ts(o_col(t), s_col(t) + p * (KT / 2) + kk * 8, vd + kk * 128, IDESC_O,
                                                    (j % FRESH > 0 || part > 0 || p < PARTS - 1 || kk > 0) ? 1u : 0u);
                                if (part == 0) {
#pragma unroll
                                    for (int i = 0; i < 2; ++i) {
                                        if (back[i] >= 0) umma_commit(&empty[back[i]]);
                                        back[i] = -1;
                                    }
                                }
                            }
                            if (!ok) continue;
                            if (j + 1 < mine)
                                scores(t, k_slot);
                            else
                                umma_commit(&o_full[t]);
                        }
                        back[0] = v_slot;
                        back[1] = j + 1 < cnt ? k_slot : -1;
                    }
                }
                umma_commit(all_done);   // every MMA is over before TMEM is released
                mbar_wait_near(all_done, 0, ta.timeout_ns, DEVERR_ATTN_WAIT);
            }
            __syncwarp();
        } else if (warp == 2) {
            // -------------------------------------------------- tiles that landed
            // V_j and K_(j+1) are in, and the value rows behind a segment's last key, which hold anything (NaN), are zeros
            // (P is zero there): an arrival on both row tiles' probability barriers
            const int end_pre = c.prefix_len % KT ? npre - 1 - j0 : -1, end_own = own_load % KT ? nall - 1 - j0 : -1;
            bool ok = true;
            for (int j = 0; ok && j < cnt; ++j) {
                const int iv = 2 * j + 1;
                if (!(ok = warp_wait(&full[iv % ST], (uint32_t)((iv / ST) & 1)))) break;
                if (j == end_pre || j == end_own) {
                    int key0;
                    const int valid = tile_keys(j0 + j, &key0);
                    const uint32_t vb = ring + (uint32_t)(iv % ST) * SM::SLOT;
                    for (int x = lane; x < (KT - valid) * 8; x += 32)
#pragma unroll
                        for (uint32_t h = 0; h < SM::HALVES; ++h)
                            st_shared_v4(vb + h * SM::HALF_KV + (uint32_t)(valid * 128 + x * 16), 0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (j + 1 < cnt && !(ok = warp_wait(&full[(iv + 1) % ST], (uint32_t)(((iv + 1) / ST) & 1)))) break;
                for (int t = 0; ok && t < 2; ++t) {
                    if (j >= (t ? cnt1 : cnt0)) continue;
                    // (this phase's arrival only once the last phase is over)
                    if (j > 0 && !(ok = warp_wait(&p_full[t], (uint32_t)((j - 1) & 1)))) break;
                    if (lane == 0) mbar_arrive(&p_full[t]);
                }
            }
        }
    } else {
        // ---------------------------------------------------------- softmax
        regs_inc<TILE_REGS_SOFTMAX>();
        const int t = (warp - 4) >> 2, quarter = warp & 3;
        const int tid = threadIdx.x & 127;          // thread of the tile's 128
        const int mine = t ? cnt1 : cnt0;
        // Q into shared memory: consecutive threads take consecutive 16 bytes of a row
        if (mine > 0) {
            constexpr int CH = D / 8, STEP = TILE_ROWS / CH, N = TILE_ROWS / STEP;
            const uint32_t qb = q_smem + t * SM::QB;
            const int ch = tid % CH, r0 = tid / CH;
            // rows r0, r0 + STEP, ...: their tokens and heads by addition, all the loads in flight at once
            const int ri = rs.row0 + t * TILE_ROWS + r0, tok_step = STEP / a.G, head_step = STEP % a.G;
            int tok = ri / a.G, head = ri % a.G;
            uint4 v[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                v[i] = make_uint4(0u, 0u, 0u, 0u);
                if (t * TILE_ROWS + r0 + i * STEP < rows)
                    v[i] = __ldg(reinterpret_cast<const uint4 *>(
                        a.q + ((size_t)(rs.tok0 + tok) * a.H + (size_t)g * a.G + head) * D + 8 * ch));
                tok += tok_step;
                head += head_step;
                if (head >= a.G) {
                    head -= a.G;
                    ++tok;
                }
            }
            const uint32_t sign = ta.flip ? 0x80008000u : 0u;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int r = r0 + i * STEP;
                st_shared_v4(qb + (ch / 8) * SM::HALF_Q + r * 128 + (((ch % 8) ^ (r & 7)) << 4), v[i].x ^ sign,
                             v[i].y ^ sign, v[i].z ^ sign, v[i].w ^ sign);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[t]);
        }
        const int r = t * TILE_ROWS + 32 * quarter + lane;   // this thread's row of the pair
        const bool live = r < rows;
        int pre = 0, own = 0;                                // keys of each segment that the row sees
        if (live) {
            if (ta.prefix_only) {
                pre = c.prefix_len;
            } else {
                own = own_seen(rs, a.G, rs.row0 + r);
                pre = own < 0 ? 0 : c.prefix_len;
            }
        }
        const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
        const uint32_t sc = s_col(t) + lane_off, oc = o_col(t) + lane_off;
        float m = -INFINITY, l = 0.f;   // m: what the exponents are taken against (see TileRange)
        // the row's place in fp32: a partial result's values, or the output's (kept is the m its sums refer to)
        float *row32 = nullptr, kept = -INFINITY;
        const int ri = rs.row0 + r;
        const size_t at = live ? ((size_t)(rs.tok0 + ri / a.G) * a.H + (size_t)g * a.G + ri % a.G) * D : 0;
        if (ta.part)
            row32 = ta.part + (((size_t)(pair * c.Hkv + g) * ta.splits + split) * PAIR_ROWS + r) * part_stride(D) + 4;
        else if (!a.out16)
            row32 = static_cast<float *>(a.out) + at;
        // with one part: what the row's place holds is in units of this
        float unit = 1.f;
        auto load_kept = [&](int x, float(&k)[8]) {
            if (ta.part || PARTS > 1) {
                const float4 u = __ldcg(reinterpret_cast<const float4 *>(row32 + x)),
                             v = __ldcg(reinterpret_cast<const float4 *>(row32 + x + 4));
                k[0] = u.x, k[1] = u.y, k[2] = u.z, k[3] = u.w;
                k[4] = v.x, k[5] = v.y, k[6] = v.z, k[7] = v.w;
            } else {
                const uint4 u = __ldcg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.out) + at + x));
                k[0] = lo16<XT>(u.x), k[1] = hi16<XT>(u.x), k[2] = lo16<XT>(u.y), k[3] = hi16<XT>(u.y);
                k[4] = lo16<XT>(u.z), k[5] = hi16<XT>(u.z), k[6] = lo16<XT>(u.w), k[7] = hi16<XT>(u.w);
            }
        };
        bool ok = true;
        int j = 0;
        while (j < mine) {
            if (PARTS == 1 && j > 0) {
                if (!(ok = all_wait(&s_full[t], (uint32_t)(j & 1)))) break;
                tc_fence_after();
                // (the tensor core is done with O, as it has formed S since.)  |O| and what is kept stay below l times
                // 65504, the largest value, so 16 bits hold their sum in units of 2 l or more; the remainder is exact
                const float f = kept == -INFINITY ? 0.f : ex2(kept - m) * unit;
                if (!ta.part) unit = __uint_as_float((__float_as_uint(l) & 0x7f800000u) + 0x01000000u);
                const float per_unit = __uint_as_float(0x7f000000u - __float_as_uint(unit));
#pragma unroll 1
                for (int x = 0; x < D; x += 32) {
                    uint32_t o[32];
                    __syncwarp();
                    tmem_ld_32x32b_x32(oc + x, o);
                    tmem_wait_ld();
                    if (live) {
#pragma unroll
                        for (int y = 0; y < 32; y += 8) {
                            float k[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                            if (j > RELIEF) load_kept(x + y, k);
#pragma unroll
                            for (int e = 0; e < 8; ++e) k[e] = fmaf(k[e], f, __uint_as_float(o[y + e]));
                            if (ta.part) {
#pragma unroll
                                for (int e = 0; e < 8; ++e) o[y + e] = 0u;
                                __stcg(reinterpret_cast<float4 *>(row32 + x + y), make_float4(k[0], k[1], k[2], k[3]));
                                __stcg(reinterpret_cast<float4 *>(row32 + x + y + 4), make_float4(k[4], k[5], k[6], k[7]));
                            } else {
                                uint32_t h[4];
#pragma unroll
                                for (int e = 0; e < 8; e += 2) {
                                    h[e / 2] = pack16<XT>(k[e] * per_unit, k[e + 1] * per_unit);
                                    o[y + e] = __float_as_uint(fmaf(lo16<XT>(h[e / 2]), -unit, k[e]));
                                    o[y + e + 1] = __float_as_uint(fmaf(hi16<XT>(h[e / 2]), -unit, k[e + 1]));
                                }
                                __stcg(reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + at + x + y),
                                       make_uint4(h[0], h[1], h[2], h[3]));
                            }
                        }
                    }
                    __syncwarp();
                    tmem_st_32x32b_x32(oc + x, o);
                }
                tmem_wait_st();
                kept = m;
            }
            for (const int end = PARTS == 1 ? min(mine, j + RELIEF) : mine; j < end; ++j) {
                if (!(ok = all_wait(&s_full[t], (uint32_t)(j & 1)))) break;
                tc_fence_after();
                const bool fresh = PARTS > 1 && j > 0 && j % FRESH == 0;
                if (fresh) {
                    // O's sums of the last tiles join those kept (the tensor core is done with O: it has formed S since).
                    // With the maximum unchanged since, as it mostly is, that is an addition in memory, which is not
                    // waited for; the row is this thread's alone, so the order of additions is fixed.
                    const float f = kept == -INFINITY ? 0.f : ex2(kept - m);
                    const int how = j == FRESH ? 0 : __all_sync(0xffffffffu, f == 1.f || !live) ? 1 : 2;
#pragma unroll 1
                    for (int x = 0; x < D; x += 32) {
                        uint32_t o[32];
                        __syncwarp();
                        tmem_ld_32x32b_x32(oc + x, o);
                        tmem_wait_ld();
                        if (!live) continue;
                        float *p = row32 + x;
#pragma unroll
                        for (int y = 0; y < 32; y += 4) {
                            float4 v = make_float4(__uint_as_float(o[y]), __uint_as_float(o[y + 1]), __uint_as_float(o[y + 2]),
                                                   __uint_as_float(o[y + 3]));
                            if (how == 1) {
                                asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p + y), "f"(v.x),
                                             "f"(v.y), "f"(v.z), "f"(v.w)
                                             : "memory");
                                continue;
                            }
                            if (how == 2) {
                                const float4 k = __ldcg(reinterpret_cast<const float4 *>(p + y));
                                v = make_float4(fmaf(k.x, f, v.x), fmaf(k.y, f, v.y), fmaf(k.z, f, v.z), fmaf(k.w, f, v.w));
                            }
                            __stcg(reinterpret_cast<float4 *>(p + y), v);
                        }
                    }
                    __syncwarp();
                    kept = m;
                }
                uint32_t s[KT];
                int key0;
                tile_keys(j0 + j, &key0);
                const int limit = (j0 + j < npre ? pre : own) - key0;   // keys of the tile that the row sees
                const bool cut = __any_sync(0xffffffffu, limit < KT);
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int x = 0; x < 64; x += 32) tmem_ld_32x32b_x32(sc + x, *reinterpret_cast<uint32_t(*)[32]>(s + x));
                tmem_wait_ld();
                // the second half's scores arrive under the first's maximum
#pragma unroll
                for (int x = 64; x < KT; x += 32) tmem_ld_32x32b_x32(sc + x, *reinterpret_cast<uint32_t(*)[32]>(s + x));
#pragma unroll
                for (int x0 = 0; x0 < KT; x0 += 64) {
                    if (x0 > 0) tmem_wait_ld();
                    if (cut) {
#pragma unroll
                        for (int x = x0; x < x0 + 64; ++x)
                            if (x >= limit) s[x] = 0xff800000u;         // -inf
                    }
#pragma unroll
                    for (int x = x0; x < x0 + 64; x += 2)
                        mx[(x / 2) & 3] = max3(mx[(x / 2) & 3], __uint_as_float(s[x]), __uint_as_float(s[x + 1]));
                }
                const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * a.qscale;
                // (the first tile with a live key sets m; O is overwritten by the first product)
                using R = TileRange<XT>;
                const float room = XT == X_F16 && fabsf(m) >= R::EXACT ? R::FAR_ROOM : R::ROOM;
                const bool grown = top > m + room || (m == -INFINITY && top > m);
                if (__any_sync(0xffffffffu, grown)) {
                    float lift = R::LIFT;
                    if constexpr (XT == X_F16) {
                        // (mx: the maxima of four interleaved quarters of the tile's keys)
                        if (top - fminf(fminf(mx[0], mx[1]), fminf(mx[2], mx[3])) * a.qscale > R::ALONE) lift = R::ALONE_LIFT;
                        if (fabsf(top) >= R::EXACT) lift = 0.f;
                    }
                    const float mn = grown ? top - lift : m;
                    const float f = grown ? ex2(m - mn) : 1.f;          // 0 while m = -inf
                    m = mn;
                    l *= f;
                    if (j > 0 && !fresh) {
#pragma unroll
                        for (int x = 0; x < D; x += 32) {
                            uint32_t o[32];
                            tmem_ld_32x32b_x32(oc + x, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                            tmem_st_32x32b_x32(oc + x, o);
                        }
                    }
                }
                const float base = m == -INFINITY ? 0.f : m;            // a row that has seen nothing: all zeros
                const uint64_t scale2 = pack2(a.qscale, a.qscale), base2 = pack2(-base, -base);
                uint64_t sum2[2] = {0, 0};
#pragma unroll
                for (int x0 = 0; x0 < KT; x0 += 32) {
                    uint32_t h[16];
#pragma unroll
                    for (int x = 0; x < 32; x += 2) {
                        const uint64_t y = fma2(pack2(__uint_as_float(s[x0 + x]), __uint_as_float(s[x0 + x + 1])), scale2, base2);
                        float p0, p1;
                        unpack2(y, p0, p1);
                        p0 = ex2(p0);
                        p1 = ex2(p1);
                        sum2[(x / 2) & 1] = add2(sum2[(x / 2) & 1], pack2(p0, p1));
                        h[x / 2] = pack16<XT>(p0, p1);
                        if constexpr (PARTS > 1) {
                            s[x0 + x] = __float_as_uint(p0 - lo16<XT>(h[x / 2]));
                            s[x0 + x + 1] = __float_as_uint(p1 - hi16<XT>(h[x / 2]));
                        }
                    }
                    tmem_st_32x32b_x16(sc + x0 / 2, h);
#pragma unroll
                    for (int p = 1; p < PARTS; ++p) {
#pragma unroll
                        for (int x = 0; x < 32; x += 2) {
                            const float r0 = __uint_as_float(s[x0 + x]), r1 = __uint_as_float(s[x0 + x + 1]);
                            h[x / 2] = pack16<XT>(r0, r1);
                            s[x0 + x] = __float_as_uint(r0 - lo16<XT>(h[x / 2]));
                            s[x0 + x + 1] = __float_as_uint(r1 - hi16<XT>(h[x / 2]));
                        }
                        tmem_st_32x32b_x16(sc + p * (KT / 2) + x0 / 2, h);
                    }
                    if (x0 + 32 == SPLIT || x0 + 32 == KT) {   // a part is ready
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&p_full[t + (x0 + 32 == KT ? 2 : 0)]);
                    }
                }
                float l0, l1;
                unpack2(add2(sum2[0], sum2[1]), l0, l1);
    l += l0 + l1;
            }
            if (!ok) break;
        }
        // ---------------------------------------------------------- results
        if (mine > 0 && ok) ok = warp_wait(&o_full[t], 0);
        tc_fence_after();
        if (ok) {
            // (scores that are not numbers leave no maximum: the merge is to see their sum, not to take the row as empty)
            if (ta.part && live) *reinterpret_cast<float2 *>(row32 - 4) = make_float2(l == l ? m : 0.f, l);
            const bool more = mine > (PARTS > 1 ? FRESH : RELIEF);   // sums were kept
            const float fk = more && kept != -INFINITY ? ex2(kept - m) * unit : 0.f;
            const float inv = ta.part ? 1.f : 1.f / l;
#pragma unroll
            for (int x0 = 0; x0 < D; x0 += 32) {
                uint32_t o[32];
                __syncwarp();
                if (mine > 0) {
                    tmem_ld_32x32b_x32(oc + x0, o);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int x = 0; x < 32; ++x) o[x] = 0u;
                }
                if (!live) continue;
                float f[32];
#pragma unroll
                for (int x = 0; x < 32; ++x) f[x] = __uint_as_float(o[x]);
                if (more) {
#pragma unroll
                    for (int x = 0; x < 32; x += 8) {
                        float k[8];
                        load_kept(x0 + x, k);
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[x + e] = fmaf(k[e], fk, f[x + e]);
                    }
                }
#pragma unroll
                for (int x = 0; x < 32; ++x) f[x] = l == 0.f ? 0.f : f[x] * inv;   // (a row that saw nothing)
                if (!ta.part && a.out16) {
                    uint16_t *dst = static_cast<uint16_t *>(a.out) + at + x0;
#pragma unroll
                    for (int x = 0; x < 32; x += 8)
                        *reinterpret_cast<uint4 *>(dst + x) =
                            make_uint4(pack16<XT>(f[x], f[x + 1]), pack16<XT>(f[x + 2], f[x + 3]),
                                       pack16<XT>(f[x + 4], f[x + 5]), pack16<XT>(f[x + 6], f[x + 7]));
                } else {
                    float *dst = row32 + x0;
#pragma unroll
                    for (int x = 0; x < 32; x += 4)
                        *reinterpret_cast<float4 *>(dst + x) = make_float4(f[x], f[x + 1], f[x + 2], f[x + 3]);
                }
            }
        }
        tc_fence_before();
    }

    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TILE_TMEM_COLS);
    }
}

// Merges the key splits of a prefill: a warp per (token, query head), its lanes
// the columns.
template <int XT, int D>
__global__ void __launch_bounds__(256) paged_tile_combine_kernel(const PagedTileArgs ta) {
    constexpr int PS = part_stride(D), E = D / 32, U = 4;
    const PagedAttnArgs &a = ta.a;
    const PagedArgs &c = a.c;
    const int lane = threadIdx.x & 31;
    const long w = (long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int t = (int)(w / a.H), hh = (int)(w % a.H), g = hh / a.G;
    if (t >= a.T) {
        pdl_wait();
        return;
    }
    // the token's sequence, and the pairs of row tiles before it
    int b = 0, tok0 = 0, n = 0;
    long before = 0;
    for (int i0 = 0; i0 < c.B; i0 += 32) {
        const int i = i0 + lane;
        const int lo = i < c.B ? first_token(a, i) : 0, k = i < c.B ? token_count(a, i) : 0;
        const unsigned hit = __ballot_sync(0xffffffffu, k > 0 && t >= lo && t < lo + k);
        const int at = hit ? __ffs(hit) - 1 : 32;
        long sum = lane < at ? pairs_of(k, a.G) : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        before += sum;
        if (hit) {
            b = i0 + at;
            tok0 = __shfl_sync(0xffffffffu, lo, at);
            n = __shfl_sync(0xffffffffu, k, at);
            break;
        }
    }
    const long ri = (long)(t - tok0) * a.G + hh % a.G;
    const long pair = before + pairs_of(n, a.G) - 1 - ri / PAIR_ROWS;
    // behind the last sequence, or of offsets that do not ascend, whose sequences overlap and have more pairs than there
    // are partial results (the wait all the same: this kernel may not end before the tiles')
    if (n == 0 || pair >= ta.pairs) {
        pdl_wait();
        return;
    }
    const int r = (int)(ri % PAIR_ROWS);
    pdl_wait();
    const float *p0 = ta.part + (((size_t)(pair * c.Hkv + g) * ta.splits) * PAIR_ROWS + r) * PS;
    float M = -INFINITY, L = 0.f, A[E];
#pragma unroll
    for (int e = 0; e < E; ++e) A[e] = 0.f;
    for (int s0 = 0; s0 < ta.splits; s0 += U) {
        float mv[U], lv[U], av[U][E];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float *p = p0 + (size_t)(s0 + u < ta.splits ? s0 + u : 0) * PAIR_ROWS * PS;
            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(p));
            mv[u] = s0 + u < ta.splits ? ml.x : -INFINITY;
            lv[u] = ml.y;
#pragma unroll
            for (int e = 0; e < E; ++e) av[u][e] = __ldcg(p + 4 + 32 * e + lane);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) merge_part(M, L, A, mv[u], lv[u], av[u]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) store_out<XT>(a, (size_t)w * D + 32 * e + lane, L == 0.f ? 0.f : A[e] / L);
}

}  // namespace lwq
