/*
 * lwq.h -- block-quantized matmul for NVIDIA B200 (sm_100a).
 *
 *     y[M,N] = x[M,K] . dequant(Wq[N,K])^T
 *
 * The weights Wq are stored in llama.cpp-style blocks (the "legacy" and
 * "K-quant" families named in "Resumo Tecnico: Llamas na Web",
 * "Declaracao do Problema" item 3, and in its "3. Design de Shader Consciente
 * de Quantizacao", which co-designs dequantization with the matmul kernels:
 * decoded in registers for the matrix-vector (decode) case and in shared
 * memory, reused across rows, for the matrix-matrix (prefill) case).
 *
 * Paths (chosen per call by a per-shape configuration table, the analogue of
 * the tunable tile sizes in "2. Biblioteca de Kernels Portatil em
 * Desempenho", "Parametros Ajustaveis"):
 *   M <= 16  decode GEMV: packed rows staged by TMA into shared memory,
 *            decoded in registers, multiplied on the tensor cores with
 *            warp-level MMAs, split-K partials reduced deterministically;
 *   M >  16  prefill GEMM: packed tiles staged by TMA, dequantized to
 *            bf16/fp16 in shared memory, tcgen05 MMAs accumulating in TMEM.
 * Q6_K rows that are not 16-byte multiples (K not a multiple of 2048) and Q2_K
 * rows (K not a multiple of 1024) stream as slots of the flat matrix (whole
 * 16-byte units per row) into both paths, which needs N * lwq_row_bytes(fmt,
 * K) to be a multiple of 16.  Shapes
 * no tensor-core path takes (K not a multiple of 256, or such a matrix that is
 * not a whole number of 16-byte units) run a simple GEMV kernel.
 *
 * Everything is plain C: pointers and sizes, no C++ or framework types.
 */
#ifndef LWQ_H
#define LWQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------ status codes */
typedef enum {
    LWQ_OK = 0,
    LWQ_ERR_INVALID_ARG = 1,        /* a size is <= 0, K is not a multiple of the block, NULL pointer */
    LWQ_ERR_UNSUPPORTED = 2,        /* unknown format / activation code, or a shape no path handles */
    LWQ_ERR_MISALIGNED = 3,         /* Wq, x, y or the workspace is not 16-byte aligned */
    LWQ_ERR_NOT_INITIALIZED = 4,    /* a call needs the workspace and lwq_init was not called on this device */
    LWQ_ERR_WORKSPACE_TOO_SMALL = 5,/* the registered workspace is smaller than this call needs */
    LWQ_ERR_CUDA = 6,               /* a CUDA runtime/driver call failed (launch error, bad device) */
    LWQ_ERR_DEVICE_TIMEOUT = 7,     /* a kernel gave up a bounded wait (see lwq_get_device_error) */
    LWQ_ERR_BAD_PAGE = 8            /* a page table held a page outside the cache (see lwq_get_device_error) */
} lwq_status;

/* ------------------------------------------------- format and dtype codes
 * fmt = weight format | activation dtype [| flags, below].
 *
 * LWQ_Q8_0: 32 weights per 34-byte block: fp16 d (little endian), int8 q[32];
 *           w = d*q.
 * LWQ_Q4_0: 32 weights per 18-byte block: fp16 d, 16 bytes b[16]; byte i
 *           holds element i in its low nibble and element i+16 in its high
 *           nibble; w = (nibble - 8)*d.
 * LWQ_Q4_K: 256 weights per 144-byte superblock: fp16 d, fp16 dmin, 12 bytes
 *           of eight 6-bit (scale, min) pairs (for j < 4: sc_j = s[j]&63,
 *           m_j = s[j+4]&63; for j >= 4: sc_j = (s[j+4]&15)|((s[j-4]>>6)<<4),
 *           m_j = (s[j+4]>>4)|((s[j]>>6)<<4)), 128 bytes of nibbles in 4
 *           groups of 32 (group g: low nibbles are sub-block 2g, high
 *           nibbles sub-block 2g+1); w = d*sc_j*q - dmin*m_j.
 * More K-quant formats of the same family ("Resumo Tecnico: Llamas na Web"
 * names q4_k_m, which mixes Q4_K and Q6_K tensors, and q2_k, without their
 * layouts; these are the llama.cpp layouts of those names):
 * LWQ_Q6_K: 256 weights per 210-byte superblock: ql[128] (low 4 bits of the
 *           6-bit codes), qh[64] (high 2 bits), int8 sc[16] (one scale per 16
 *           weights), fp16 d.  Element 128n+32g+l (n<2, g<4, l<32) takes
 *           nibble g>>1 of ql[64n+32(g&1)+l] and bits 2g, 2g+1 of qh[32n+l];
 *           w = d*sc[e/16]*(q - 32).
 * LWQ_Q5_K: 256 weights per 176-byte superblock: fp16 d, fp16 dmin, the 12
 *           scale/min bytes of Q4_K, qh[32], qs[128].  Element 64g+32h+l
 *           takes nibble h of qs[32g+l] and (as bit 4) bit 2g+h of qh[l];
 *           w = d*sc_j*q - dmin*m_j, j = 2g+h.
 * LWQ_Q2_K: 256 weights per 84-byte superblock: s[16] (per 16 weights: scale
 *           in the low nibble, min in the high nibble), qs[64], fp16 d, fp16
 *           dmin.  Element 128n+32j+l takes bits 2j, 2j+1 of qs[32n+l];
 *           w = d*(s[e/16]&15)*q - dmin*(s[e/16]>>4).
 * Activations x: fp32, fp16 or bf16, row-major [M][K].
 */
#define LWQ_Q8_0 1
#define LWQ_Q4_0 2
#define LWQ_Q4_K 3
#define LWQ_Q6_K 4
#define LWQ_Q5_K 5
#define LWQ_Q2_K 6
#define LWQ_FMT_MASK 0xFF
#define LWQ_ACT_F32 0x000
#define LWQ_ACT_F16 0x100
#define LWQ_ACT_BF16 0x200
#define LWQ_ACT_MASK 0xF00
/* Optional flag, or-ed into fmt: the caller promises that Wq is not written
 * by any work still running on the stream when the call is made (weights are
 * constant, as in a decode loop).  The call's kernels are then launched as
 * programmatic dependent launches: they may start, and begin streaming Wq,
 * before the preceding kernel on the stream has finished; they still wait for
 * it to complete before reading x or writing y and the workspace.  This hides
 * launch latency between back-to-back calls. */
#define LWQ_FLAG_OVERLAP 0x1000
/* Optional flag, or-ed into fmt: int8 activation blocks ("quantized arithmetic
 * without runtime dequantization", "Compute Shaders con WebGPU para Inferencia
 * ML").  Each run of 32 activations of a row (K must be a multiple of 256) is
 * quantized in the kernel to int8 codes q with one fp32 scale d, per block in
 * fp32 with round-to-nearest-even:
 *   amax = max |x|;  amax < 2^-100: d = 0, q = 0;  else d = amax / 127,
 *   q = rint(x * (127 / amax)),
 * 16-bit activations first widened exactly; and y = x_q * dequant(Wq)^T with
 * x_q = q * d, the block dot products taken in integers (s8 x s8 -> s32) and
 * scaled in fp32.  Results differ from the unquantized product by the
 * activation rounding (max |y - y_exact| / sum |x w| stays below 1e-2 for
 * N(0,1) activations); against x_q they agree to fp32 rounding.  Supported for
 * Q4_0, Q8_0 and Q4_K weights at any M, in passes of 8 activation rows (each pass
 * streams the weights: a prefill-sized M reads them M/8 times); other formats
 * return LWQ_ERR_UNSUPPORTED.  Activations must be finite. */
#define LWQ_FLAG_ACT_I8 0x2000

/* Bytes of one packed row of K weights (K/32*34, K/32*18, K/256*144,
 * K/256*210, K/256*176, K/256*84), or 0
 * when fmt is unknown or K is not a positive multiple of the block size. */
size_t lwq_row_bytes(int fmt, int64_t K);

/* Device workspace bytes that lwq_matmul needs for every call with
 * M <= max_M, N <= max_N, K <= max_K in this format.  The workspace holds the
 * split-K partial sums (fp32), which a follow-up kernel adds in split order
 * (deterministic); it is the library's one static arena,
 * sized once at start-up ("1. Inferencia Local Eficiente em Memoria",
 * "Alocacao Estatica de Memoria" and "Arena de Buffer de Parametros").
 * Returns 0 for invalid arguments. */
size_t lwq_workspace_size(int fmt, int max_M, int max_N, int max_K);

/* Register the caller-owned device workspace for the CURRENT device.
 * d_workspace: device pointer, 16-byte aligned (NULL with bytes == 0 is
 * allowed: calls that need no workspace still run).  The library keeps the
 * pointer until lwq_shutdown or the next lwq_init on this device; it never
 * allocates, frees or reads it outside lwq_matmul, and its contents need no
 * initial value.  No device work is done here.  Errors: LWQ_ERR_MISALIGNED,
 * LWQ_ERR_INVALID_ARG, LWQ_ERR_CUDA (no current device). */
int lwq_init(void *d_workspace, size_t bytes);

/* Forget the workspace registered for the current device.  Always LWQ_OK. */
int lwq_shutdown(void);

/*
 * y[M,N] (fp32, row-major) = x[M,K] . dequant(Wq)^T.
 *
 *   fmt     weight format | activation dtype, optionally | LWQ_FLAG_OVERLAP
 *           and | LWQ_FLAG_ACT_I8 (codes above)
 *   Wq      device pointer, N packed rows of lwq_row_bytes(fmt, K) bytes each
 *   x       device pointer, row-major [M][K] in the activation dtype
 *   y       device pointer, row-major [M][N] fp32, fully overwritten
 *   M, N, K sizes (> 0); K a multiple of 32 (Q8_0, Q4_0) or 256 (K-quants)
 *   stream  a cudaStream_t (NULL = the legacy default stream)
 *
 * Ownership: the caller owns Wq, x, y and the workspace.  The call is
 * asynchronous: it validates the arguments on the host, enqueues its
 * kernels on `stream` (one per pass of activation rows, plus a split-K sum
 * kernel per pass when K is split; lwq_last_launch_count tells how many) and
 * returns; it never allocates and never synchronizes
 * the host.  Kernel faults surface at the caller's next synchronization, as
 * with any CUDA launch.  Wq, x and y must be 16-byte aligned
 * (LWQ_ERR_MISALIGNED).  Calls that use split-K (see lwq_workspace_size) need
 * a registered workspace (LWQ_ERR_NOT_INITIALIZED,
 * LWQ_ERR_WORKSPACE_TOO_SMALL); calls sharing one workspace must be ordered
 * (one stream, or events), since their partial sums share the arena.  A GEMV
 * call whose chosen plan splits K but finds too little workspace takes the
 * plan with a warp per chunk of K instead when that one needs no more (the
 * K-quants with 9..16 rows of 16-bit x or 3..5 of fp32 x and K <= 4096), so it
 * runs as it would with no workspace; lwq_workspace_size covers the faster plan.
 * M > 16 with fp32 activations runs the GEMV path over groups of rows of x.
 */
int lwq_matmul(int fmt, const void *Wq, const void *x, float *y, int M, int N, int K, void *stream);

/* lwq_matmul for callers that cannot allocate device memory: code that may
 * not call the CUDA allocator (an allocator's own callbacks, a process whose
 * memory pool is fixed and fully handed out at start-up, a plugin given only
 * input and output pointers).  It needs no workspace and no lwq_init: its
 * split-K scratch is a static 4 MiB device array inside the library, held on
 * every device that loads the library until the process exits.  The pages
 * this library follows have no counterpart of this entry point.
 *
 * Arguments, layouts and results are those of lwq_matmul.  Only the decode
 * GEMV is offered: M <= 16 and the shapes lwq_select_config sends to path 1,
 * else LWQ_ERR_UNSUPPORTED.  A shape whose split-K scratch
 * (lwq_workspace_size bytes) exceeds 4 MiB returns LWQ_ERR_WORKSPACE_TOO_SMALL.
 * The first call on a device looks up the array's device address (make it
 * before any stream capture).  Calls share the array, which needs no initial
 * value; calls whose kernels overlap on the GPU race.  Nothing is allocated
 * or freed. */
int lwq_matmul_noalloc(int fmt, const void *Wq, const void *x, float *y, int M, int N, int K, void *stream);

/* ------------------------------------------------ configuration table
 * The per-shape configuration lwq_matmul would use, and a way to force one
 * (used by the sweep that fills the table and by tests). */
typedef struct {
    int path;        /* 1 = GEMV (tensor-core MMA), 2 = GEMM (tcgen05), 3 = simple GEMV */
    int warps;       /* GEMV: compute warps per CTA, each owning 256 weights of K */
    int stages;      /* pipeline depth (shared-memory ring stages) */
    int splits;      /* GEMV: split-K factor (1 = none) */
    int ctas;        /* CTAs launched (persistent grid) */
    int tile_n;      /* GEMM: output columns per tile (weight rows): 128, or 256 as two
                        128-row halves sharing each activation tile */
    int tile_m;      /* GEMM: output rows per tile (activation rows) */
    int reserved[5];
} lwq_config;

/* Fill *cfg with the configuration lwq_matmul(fmt, ., ., ., M, N, K) would
 * use on the current device.  Errors as lwq_matmul's argument checks. */
int lwq_select_config(int fmt, int M, int N, int K, lwq_config *cfg);

/* lwq_matmul with a forced configuration.  Fields set to 0 take the table's
 * value; an impossible configuration returns LWQ_ERR_UNSUPPORTED. */
int lwq_matmul_config(int fmt, const void *Wq, const void *x, float *y, int M, int N, int K,
                      const lwq_config *cfg, void *stream);

/* ------------------------------------------------------ decode attention
 * One query token per sequence and head against that sequence's key/value
 * cache, the softmax fused into the one pass over the keys ("Compute Shaders
 * con WebGPU para Inferencia ML", "El Mecanismo de Atencion": scores
 * q.k / sqrt(head_dim), a running maximum and sum, the weighted values
 * accumulated in the same pass):
 *   s_j = scale * (q . k_j),  out = sum_{j < len} softmax(s)_j v_j.
 * dtype: LWQ_ACT_F16 or LWQ_ACT_BF16, the type of q, k and v.
 * q [B][H][D]; k, v [B][Hkv][Lmax][D] (the caches, key j of sequence b and kv
 * head g at [b][g][j]); out [B][H][D] fp32; all row-major device arrays,
 * 16-byte aligned.  Query head h reads kv head h / (H / Hkv); H / Hkv must be
 * 1, 2, 4 or 8, and D 64 or 128.  seq_lens: device array of B int32 lengths
 * (a length outside [1, Lmax] is clamped into it), or NULL for Lmax each.
 * scale: usually 1 / sqrt(D).  Long sequences are split over several CTAs
 * whose partial results a second kernel merges; the partials live in the
 * workspace registered with lwq_init (the static arena that "Llamas na Web",
 * "Alocacao Estatica de Memoria", sizes at start-up for FlashAttention-style
 * scratch), lwq_attention_workspace_size bytes.  Errors: LWQ_ERR_INVALID_ARG
 * (a size <= 0, H not a multiple of Hkv, NULL q/k/v/out, non-finite scale),
 * LWQ_ERR_UNSUPPORTED (dtype, D, H / Hkv), LWQ_ERR_MISALIGNED,
 * LWQ_ERR_NOT_INITIALIZED / LWQ_ERR_WORKSPACE_TOO_SMALL (split partials),
 * LWQ_ERR_CUDA.  The library allocates nothing and does not synchronize. */
size_t lwq_attention_workspace_size(int B, int H, int Hkv, int Lmax, int D);
int lwq_attention_decode(int dtype, const void *q, const void *k, const void *v, const int32_t *seq_lens, float *out,
                         int B, int H, int Hkv, int Lmax, int D, float scale, void *stream);

/* ------------------------------------------------------ paged key/value cache
 * The operators between the qkv projection and the output projection of a
 * serving step, over one cache that many sequences share:
 *   lwq_kv_append           rotate q and k by position, store k and v
 *   lwq_attention_paged     one query token per sequence (decode), with the
 *                           tokens that all sequences begin with read once
 *   lwq_attention_prefill   several new tokens per sequence, causally
 *
 * lwq_paged describes the cache and one batch of sequences:
 *   k, v       [num_pages][Hkv][page][D] in dtype, 16-byte aligned
 *   tables     [B][max_pages] int32, device: the page of tokens page * i ..
 *              page * i + page - 1 of each sequence.  Entries past a
 *              sequence's length are not read.
 *   lens       [B] int32, device: tokens of each sequence in the cache, those
 *              that the call appends or attends with included, the shared
 *              prefix not.  0 (or less) is an empty sequence, e.g. a padded
 *              row of a captured batch.  The attention calls take a length
 *              beyond max_pages * page as max_pages * page (so the last new
 *              token sees all of the table's tokens, the one before it one
 *              less); lwq_kv_append drops what lies beyond (below).
 *   prefix     [ceil(prefix_len / page)] int32, device: the pages of a prefix
 *              that every sequence begins with (a system prompt); NULL with
 *              prefix_len 0.  Token j of a sequence is then at position
 *              prefix_len + j.
 *   dtype      LWQ_ACT_F16 or LWQ_ACT_BF16, of the cache and of q
 *   D          64 or 128;  page: 16, 32, 64, 128 or 256
 * The caller owns all of it; the struct itself is read during the call only.
 * A page number outside [0, num_pages) that a live token needs is never
 * followed: its keys and values read as zeros, nothing is stored for it, and
 * lwq_get_device_error then returns LWQ_ERR_BAD_PAGE.  Memory in pages behind
 * a sequence's last token may hold anything, NaN included. */
typedef struct {
    void *k, *v;
    const int32_t *tables;
    const int32_t *lens;
    const int32_t *prefix;
    int prefix_len;
    int dtype;
    int B, Hkv, D, page, max_pages, num_pages;
} lwq_paged;

/* Rotary positions.  Pair i of a head (i < rot_dim / 2) turns by the angle
 * position[axis(i)] * f_i:  (a, b) -> (a cos - b sin, b cos + a sin); the
 * elements from rot_dim on stay.
 *   LWQ_ROPE_HALF   pair i is elements (i, i + rot_dim / 2)
 *   LWQ_ROPE_PAIRS  pair i is elements (2 i, 2 i + 1)
 * Angles are kept as 64-bit fractions of a full turn (f_i / (2 pi) modulo 1,
 * rounded to 2^-64), so that the product with any 32-bit position is reduced
 * exactly: cos and sin to about 2^-22, however far the position and however
 * large f_i. */
#define LWQ_ROPE_HALF 0
#define LWQ_ROPE_PAIRS 1
typedef struct {
    int rot_dim, layout, axes, reserved;
    uint64_t turn[64];      /* f_i / (2 pi) modulo 1, in units of 2^-64 */
    uint8_t axis[64];
} lwq_rope;

/* Fill *rope on the host (once; it holds no pointers and may be copied).
 *   rot_dim   a multiple of 16, 16 .. 128
 *   f_i       inv_freq[i] (rot_dim / 2 finite doubles of at most 2^20 in size),
 *             or, with inv_freq NULL, base^(-2 i / rot_dim), base > 0, in 64
 *             bits, which is off by too much at far positions where it exceeds
 *             256: refused, LWQ_ERR_INVALID_ARG
 *   axes      1 .. 4 position axes (3 for time, height and width); sections:
 *             how many consecutive pairs each axis turns, rot_dim / 2 in all
 *             (NULL with one axis)
 * Errors: LWQ_ERR_INVALID_ARG, LWQ_ERR_UNSUPPORTED (rot_dim, layout, axes). */
int lwq_rope_init(lwq_rope *rope, int rot_dim, int layout, double base, const double *inv_freq, int axes,
                  const int *sections);

/* Append the k and v of T tokens to the cache, and rotate q and k on the way.
 *   rope       NULL: nothing is rotated
 *   src        LWQ_ACT_F32, _F16 or _BF16: the type of q, k and v (fp32 is
 *              what lwq_matmul writes)
 *   q          T rows of H heads, ldq elements from row to row; k, v: T rows
 *              of Hkv heads, ldk and ldv apart.  (One fused projection y of
 *              [T][(H + 2 Hkv) D]: q = y, k = y + H D, v = y + (H + Hkv) D,
 *              all three strides (H + 2 Hkv) D.)
 *   q_out      [T][H][D] in the cache's dtype; may not overlap the inputs or
 *              the cache (nor may the rows of k and v overlap the places that
 *              the call stores to).
 *              q and q_out may both be NULL: keys and values only (H is
 *              checked all the same).
 *   cu_tokens  [B + 1] int32, device, ascending from 0: sequence b's tokens
 *              are cu_tokens[b] .. cu_tokens[b + 1] - 1, the last ones of its
 *              lens[b] tokens.  NULL: one token per sequence (T == B).
 *   positions  [axes][T] int32, device, any values; NULL: prefix_len + the
 *              token's place among its sequence's lens[b], on every axis
 * Arithmetic is fp32, each result rounded once to nearest (so a value past
 * fp16's range becomes infinite there).  Tokens from cu_tokens[B] on, and
 * tokens whose place in the cache would be negative (lens[b] 0), are padding:
 * nothing is written for them.  A place beyond max_pages * page is
 * reported as LWQ_ERR_BAD_PAGE and its k and v are dropped.  Two tokens of a
 * call may not share a place in the cache (which of them stays would be open).
 * One kernel, no workspace.
 * Errors: LWQ_ERR_INVALID_ARG (sizes, NULL pointers, T != B without
 * cu_tokens, a stride below its row, q_out over an input or the cache),
 * LWQ_ERR_UNSUPPORTED (types, D, page, H / Hkv > 16, rot_dim > D, sizes past
 * 31 bits), LWQ_ERR_MISALIGNED (pointers or row strides that are not 16-byte
 * multiples; index arrays: 4 bytes), LWQ_ERR_CUDA. */
int lwq_kv_append(const lwq_paged *cache, const lwq_rope *rope, int src, const void *q, int64_t ldq, const void *k,
                  int64_t ldk, const void *v, int64_t ldv, void *q_out, const int32_t *cu_tokens,
                  const int32_t *positions, int T, int H, void *stream);

/* Flag of the two attention calls below: out in the cache's 16-bit type
 * instead of fp32.
 * Precision, relative to sum_j softmax(s)_j |v_j| and beside the rounding of
 * the scores in fp32:
 *   fp32 results     1e-6 from lwq_attention_paged's own tokens; up to 1e-5 from
 *                    a prefix's and in lwq_attention_prefill, at any length
 *   16-bit results   half a step of the type for the result's rounding.  A
 *                    prefix's tokens and lwq_attention_prefill take each weight
 *                    softmax(s)_j rounded to the type as well: up to half a step
 *                    more, as much again as the result's rounding on average
 *                    (ask for fp32 where that is too much)
 * In an fp16 cache each weight is off by up to 2^-35 of its row's largest
 * besides (lwq_attention_paged's own tokens, and where one key stands alone far
 * above the others: 2^-40).  Scores may be 1e8 in size. */
#define LWQ_FLAG_OUT16 0x4000

/* Decode attention over the paged cache: q [B][H][D] in the cache's dtype,
 * out [B][H][D] fp32 (or 16-bit, flags above).  Query h reads kv head
 * h / (H / Hkv), H / Hkv at most 16.  With s_j = scale * (q . k_j) over the
 * prefix_len + lens[b] tokens of sequence b,  out = sum_j softmax(s)_j v_j;
 * a sequence with no token at all gets zeros, a query that holds NaN gets NaN.
 * The prefix's keys and values are read once for the whole batch, as one matrix
 * product over all B queries.
 * Needs the workspace of lwq_init: lwq_attention_paged_workspace_size bytes,
 * which depends on the sizes in *cache (its pointers are not read) and never
 * on the sequences' lengths, and is enough for every call with no more
 * sequences, pages per sequence and prefix tokens.  Like lwq_matmul's, calls
 * sharing it must be ordered (one stream, or events).
 * lwq_attention_paged_workspace_size returns 0 for invalid sizes.  The keys and
 * values of live tokens must be finite.
 * Errors as lwq_kv_append's, LWQ_ERR_INVALID_ARG for a scale that is not finite
 * and for an out that overlaps q (there is no in-place form) or the cache,
 * LWQ_ERR_NOT_INITIALIZED and LWQ_ERR_WORKSPACE_TOO_SMALL. */
size_t lwq_attention_paged_workspace_size(const lwq_paged *cache, int H);
int lwq_attention_paged(const lwq_paged *cache, int flags, const void *q, void *out, int H, float scale,
                        void *stream);

/* Causal attention of several new tokens per sequence over the cache that
 * already holds them (call lwq_kv_append first): q and out [T][H][D], the
 * tokens of sequence b at cu_tokens[b] .. cu_tokens[b + 1] - 1 (NULL: one
 * each, T == B).  The token at place j of its sequence (0 .. lens[b] - 1)
 * sees the prefix and the tokens 0 .. j.  A token that sees nothing gets
 * zeros; rows from cu_tokens[B] on are left as they were.  The values of the
 * sequence's later tokens must be finite too: a token's probability of 0 for
 * them multiplies their values.  Workspace and errors as
 * lwq_attention_paged; it is needed only when few tokens meet long caches
 * and the keys are split, and lwq_attention_prefill_workspace_size bytes are
 * enough for every call with no more tokens, sequences, pages per sequence and
 * prefix tokens. */
size_t lwq_attention_prefill_workspace_size(const lwq_paged *cache, int T, int H);
int lwq_attention_prefill(const lwq_paged *cache, int flags, const void *q, void *out, const int32_t *cu_tokens,
                          int T, int H, float scale, void *stream);

/* ------------------------------------------------ errors and diagnostics */

/* Static description of a status code. */
const char *lwq_status_string(int status);

/* Device-side error word of the current device: every wait in the kernels
 * (on an mbarrier or a TMEM handoff) is bounded, in lwq_matmul and
 * lwq_matmul_noalloc alike; a kernel
 * that gives up sets a bit here and returns instead of hanging.  The paged
 * cache's kernels set another for a page number outside the cache.  The caller
 * must synchronize first.  Returns LWQ_OK, LWQ_ERR_DEVICE_TIMEOUT or
 * LWQ_ERR_BAD_PAGE (and clears the word; a timeout comes first), or
 * LWQ_ERR_CUDA. */
int lwq_get_device_error(void);

/* Launch a one-CTA kernel on `stream` that waits on an mbarrier nothing ever
 * arrives at, with a wait bound of timeout_us microseconds, so that callers
 * can check that bounded waits end and report LWQ_ERR_DEVICE_TIMEOUT through
 * lwq_get_device_error.  Faults nothing and hangs nothing. */
int lwq_selftest_timeout(unsigned timeout_us, void *stream);

/* Number of kernels the last successful lwq_matmul, lwq_matmul_config,
 * lwq_kv_append or attention call on this thread enqueued. */
int lwq_last_launch_count(void);

/* Library version, e.g. 0x000100 for 0.1.0. */
int lwq_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LWQ_H */
