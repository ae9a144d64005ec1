/*
 * pn.h - C ABI of the PN decode GEMV library for AMD Instinct MI355X (gfx950).
 *
 * The PN weight format (tensorless, "Why a P100-native weight format"):
 *   - "Every block is 34 bytes": an fp16 scale d (2 bytes) followed by eight
 *     32-bit code words.  pn3t packs ten 3-bit codes per word (80 weights per
 *     block); pn4t packs eight 4-bit codes per word (64 weights per block).
 *     A row is made of whole blocks, so K is a multiple of 80 or 64.
 *   - "Codes never straddle the two halves of a word": even codes sit in the
 *     low 16 bits, odd codes in the high 16 bits, at the same offsets.
 *   - "Exact decode in fp32": weight = d * (n - z), exact in binary32.
 *   - "Zero is a code, and the scale has a sign": z = 4 for pn3t (range
 *     -4..+3 steps); this library takes z = 8 for pn4t (-8..+7).
 * Bit layout fixed by this library where the page is silent: scale at bytes
 * 0-1 and word i at bytes 2+4i..5+4i, little-endian; word i holds the
 * block's weights C*i .. C*i+C-1 (C = 10 or 8); weight j of a word sits in
 * half (j & 1) at bit offset b*(j >> 1) from that half's lowest bit; pn3t
 * bits 15 and 31 are ignored.
 *
 * Memory: every pointer is a DEVICE pointer owned by the caller (e.g. a torch
 * tensor's data_ptr()).  Weight matrices are N rows of K/W blocks, rows
 * contiguous (row stride pn_row_bytes(t, K)); the base only needs 2-byte
 * alignment.  Activations are IEEE fp16, 4-byte aligned; outputs are fp32,
 * 4-byte aligned, overwritten (never accumulated).
 *
 * Streams: `stream` is a hipStream_t (NULL = the default stream).  Calls
 * enqueue work and return without synchronising; device faults surface at
 * the caller's next synchronisation.  The calls allocate nothing (except
 * the group-create calls, documented there).
 *
 * Threads: the calls may be made from several host threads at once, with
 * two exceptions.  A group plan must not run concurrently with itself (two
 * runs of one plan on different streams, or graph launches of it that
 * overlap): some plans keep tile counters in the plan's device memory, and
 * two runs sharing them would each compute only part of the output.  (Such
 * runs still end: each wave or workgroup stops after more steps than any
 * correct run takes, and the outputs are then unspecified.)  And a
 * plan must not be destroyed while another thread runs it.  The kernel
 * selections (pn_set_gemv_kernel, pn_set_smallm_math) belong to the calling
 * host thread, and the variant census (pn_last_variant) too.  Per-device
 * facts the library caches (compute-unit count, occupancy, raised LDS
 * limits) are filled once, under a lock.
 *
 * Errors: arguments are checked on the host before any launch; a failing
 * check returns a negative pn_status and enqueues nothing.
 */
#ifndef PN_H
#define PN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { PN_PN3T = 0, PN_PN4T = 1 } pn_type;

typedef enum {
    PN_OK = 0,
    PN_EINVAL = -1,       /* null pointer, unknown type, bad count          */
    PN_ESHAPE = -2,       /* N < 1, K not a positive multiple of W, M/ld bad */
    PN_EALIGN = -3,       /* W not 2-aligned, x/X/y/Y not 4-aligned         */
    PN_EUNSUPPORTED = -4, /* shape outside what the kernels support         */
    PN_ELAUNCH = -5,      /* the HIP launch or a HIP runtime call failed    */
    PN_ENOMEM = -6        /* device allocation failed (pn_group_create)     */
} pn_status;

/* Weights per block: 80 (pn3t) or 64 (pn4t); 0 for an unknown type. */
int pn_weights_per_block(pn_type t);

/* Bytes of one packed row of K weights: (K / W) * 34, or 0 if K is not a
 * positive multiple of W. */
size_t pn_row_bytes(pn_type t, int64_t K);

/* y[r] = sum_k w[r,k] * x[k] for r < N.
 * "One lane, one word" and "Exact decode in fp32" on the pn-format page
 * describe the decode GEMV this computes: weights decoded exactly as
 * d * (n - z), products accumulated in fp32 (any order; the result is within
 * 1e-5 * sum_k |w[r,k] x[k]| of the exact value, row by row).
 *   W : N * pn_row_bytes(t, K) bytes, 2-byte aligned
 *   x : K fp16 values, 4-byte aligned
 *   y : N fp32 values, 4-byte aligned, overwritten */
pn_status pn_gemv(pn_type t, const void *W, int64_t N, int64_t K,
                  const void *x, float *y, void *stream);

/* Two matrices of the same type and shape against one activation, one
 * launch (the fused gate + up projection of a decoder layer):
 * y0 = W0 x, y1 = W1 x.  Arguments as for pn_gemv. */
pn_status pn_gemv2(pn_type t, const void *W0, const void *W1, int64_t N,
                   int64_t K, const void *x, float *y0, float *y1, void *stream);

/* Small-batch product for M <= 16 activation rows (speculative-decoding
 * verification width M = k + 1; v100-skinny README, "How QPN works"):
 * Y[m*ldy + r] = sum_k w[r,k] * X[m*ldx + k] for m < M, r < N.
 * Each weight is decoded exactly once and used M times; products accumulate
 * in fp32, within 1e-5 * sum_k |w[r,k] X[m,k]| of the exact value.
 *   X : M rows of fp16, leading dimension ldx >= K (elements), 4-byte aligned,
 *       ldx even
 *   Y : M rows of fp32, leading dimension ldy >= N (elements), overwritten
 *   M : 1..16
 * The arithmetic unit is the one pn_set_smallm_math selected.  With MFMA,
 * rows of whole 8-block periods (K a multiple of 640 for pn3t, 512 for pn4t)
 * and a 16-byte-aligned W are streamed into LDS by DMA (kernel gemm_rows)
 * unless pn_set_gemv_kernel chose PN_GEMV_STREAM; other problems, and the
 * VALU arithmetic, use register loads (gemm_stream).  Same accuracy bar. */
pn_status pn_gemm_smallm(pn_type t, const void *W, int64_t N, int64_t K,
                         const void *X, int64_t ldx, int M,
                         float *Y, int64_t ldy, void *stream);

/* Prefill: the same product for any number of activation rows (a prompt's
 * tokens),
 *   Y[m*ldy + r] = sum_k w[r,k] X[m*ldx + k],  m < M,  w = d * (n - z),
 * with the weights decoded inside the GEMM from the packed rows and never
 * written out (the pages' engine dequantizes PN weights for a chunked
 * prefill GEMM, "What the fork adds").  Products on MFMA in fp32, each
 * block's partial sum scaled by its d in fp32; within the tolerance above.
 *   W : packed rows, 4-byte aligned; K an even number of blocks (a multiple
 *       of 160 for pn3t, 128 for pn4t), else PN_EUNSUPPORTED
 *   X : M rows of fp16, 16-byte aligned, ldx >= K and a multiple of 8
 *   Y : M rows of fp32, 4-byte aligned, ldy >= N, overwritten
 *   M : >= 1 (at most 8,388,480)
 * Allocates nothing; enqueued on `stream`. */
pn_status pn_gemm_prefill(pn_type t, const void *W, int64_t N, int64_t K,
                          const uint16_t *X, int64_t ldx, int64_t M,
                          float *Y, int64_t ldy, void *stream);

/* Arithmetic of the small-batch kernels.  Both read the weights the same way
 * and agree within the tolerance above:
 *   PN_SMALLM_MFMA  decoded weights feed matrix-core products
 *                   (v_mfma_f32_16x16x16_f16 / 16x16x32_f16), one per block
 *                   and 16 rows, each scaled by its block's d in fp32; the
 *                   default (faster on MI355X at M = 8: 3.0 vs 5.9 ms per
 *                   64-layer token);
 *   PN_SMALLM_VALU  per-lane fp16 dot products (v_dot2_f32_f16) reduced
 *                   across the lanes of a row.
 * The setting belongs to the calling host thread (every thread starts with
 * PN_SMALLM_MFMA) and is read when that thread makes a call or creates a
 * group (a group keeps the choice it was created with).  Returns PN_EINVAL
 * for an unknown value. */
typedef enum { PN_SMALLM_MFMA = 0, PN_SMALLM_VALU = 1 } pn_smallm_math;
pn_status pn_set_smallm_math(pn_smallm_math m);
pn_smallm_math pn_get_smallm_math(void);

/* Which kernel runs the M = 1 products (pn_gemv, pn_gemv2 and pn_group_*;
 * for the small-batch products see pn_gemm_smallm):
 *   PN_GEMV_AUTO    the row-tile kernel where it applies and the launch is
 *                   large enough, else the register-pipeline kernel; the
 *                   default.  The row-tile kernel applies to rows of whole
 *                   8-block periods (K a multiple of 640 for pn3t, 512 for
 *                   pn4t) with 16-byte-aligned W and x; "large enough" is at
 *                   least 32 sixteen-row tiles per compute unit (8192 tiles,
 *                   131,072 rows, on a 256-CU MI355X), because one or two
 *                   problems are split among its waves in whole tiles;
 *   PN_GEMV_STREAM  always the register-pipeline kernel;
 *   PN_GEMV_ROWS    the row-tile kernel wherever it applies, whatever the
 *                   launch size.
 * All meet the same accuracy bar.  The setting belongs to the calling host
 * thread (every thread starts with PN_GEMV_AUTO) and is read when that
 * thread makes a call or creates a group.  Returns PN_EINVAL for an unknown
 * value. */
typedef enum { PN_GEMV_AUTO = 0, PN_GEMV_STREAM = 1, PN_GEMV_ROWS = 2 } pn_gemv_kernel;
pn_status pn_set_gemv_kernel(pn_gemv_kernel k);
pn_gemv_kernel pn_get_gemv_kernel(void);

/* Dense fp32 copy of the decoded weights, out[r*K + k] = d * (n - z),
 * bit-exact with the format's definition ("Exact decode in fp32": no
 * rounding in decode, so every correct decoder gives the same bits).
 *   out : N * K fp32, 4-byte aligned */
pn_status pn_dequantize(pn_type t, const void *W, int64_t N, int64_t K,
                        float *out, void *stream);

/* Blockwise Hadamard rotation of fp16 activations (tensorless, "How
 * Qwen3.8-27B-PN3 uses it": the model's engine rotates the activations that
 * reach the PN weights at run time; the page gives no size or scale, and
 * the reading here is the one the CPU oracle fixes):
 *   out[m*ldo + b*1024 + i] =
 *       fp16_rne( sum_j H[i][j] x[m*ldx + b*1024 + j] / 32 ),
 *   H[i][j] = (-1)^popcount(i & j)   (Sylvester order, 1024 x 1024),
 * for every row m < M and every 1024-element block b of the K columns.
 * Exact up to the one fp16 rounding (ties to even; an exact zero is +0), so
 * every correct implementation gives the same bits.
 *   x, out : fp16, device, 4-byte aligned, ldx and ldo even and >= K.
 *            out may be x (same ld): rotation in place.  Other overlaps are
 *            not allowed.
 *   K      : a multiple of 1024 (else PN_ESHAPE); M >= 1.
 * Enqueued on `stream`; returns without waiting. */
#define PN_ROTATE_BLOCK 1024
pn_status pn_rotate(const uint16_t *x, int64_t K, int M, int64_t ldx,
                    uint16_t *out, int64_t ldo, void *stream);

/* A group of independent GEMVs run by one kernel launch (a decoder layer's
 * projections, or a whole per-token weight sweep).  Each entry is one
 * pn_gemv problem; the entries may mix types and shapes. */
typedef struct pn_gemv_desc {
    const void *W;   /* packed rows, device          */
    const void *x;   /* fp16 [K], device             */
    float *y;        /* fp32 [N], device, overwritten */
    int64_t N;
    int64_t K;
    int32_t type;    /* pn_type                      */
    int32_t flags;   /* 0, or PN_DESC_ROTATE         */
} pn_gemv_desc;

/* Entry flag: x is in the model's unrotated basis; the plan multiplies by
 * pn_rotate's image of x (y = W H x).  Needs K a multiple of 1024.  The plan
 * keeps a device copy of each such x, rotated at the start of every run by
 * one extra launch ahead of the GEMV launch, on the same stream. */
#define PN_DESC_ROTATE 1

typedef struct pn_group pn_group;

/* Validate `count` descriptors (host array) and build a launch plan.  This
 * call allocates device memory for the plan's tables (and for the rotated
 * copies of PN_DESC_ROTATE inputs) and copies them there synchronously; the plan holds the descriptors' device pointers, which must
 * stay valid while the plan is used.  Returns PN_ENOMEM if allocation fails.
 * The plan runs on the row-tile kernel if that takes every problem and the
 * launch (see pn_set_gemv_kernel); otherwise every problem's rows must be
 * whole groups of 8 blocks (K a multiple of 640 for pn3t, 512 for pn4t) with
 * 2*K <= 64 KiB of activation, and other shapes return PN_EUNSUPPORTED
 * (pn_gemv takes them one at a time).  The kernel choice is made here, once,
 * for the device current at this call, and the plan's tables are placed in
 * that device's memory: pn_group_run returns PN_EUNSUPPORTED when another
 * device is current.  A plan must not run concurrently with itself (see
 * "Threads" above). */
pn_status pn_group_create(const pn_gemv_desc *descs, int count, pn_group **out);

/* The small-batch counterpart: each entry is one pn_gemm_smallm problem
 * (arguments and checks as there), all run by one launch.  Any K is taken.
 * Allocation and lifetime as for pn_group_create. */
typedef struct pn_gemm_desc {
    const void *W;   /* packed rows, device                     */
    const void *X;   /* fp16 [M][ldx], device                   */
    float *Y;        /* fp32 [M][ldy], device, overwritten      */
    int64_t N;
    int64_t K;
    int64_t ldx;     /* elements, >= K, even                    */
    int64_t ldy;     /* elements, >= N                          */
    int32_t type;    /* pn_type                                 */
    int32_t M;       /* 1..16 (pn_gemm_prefill_group: >= 1)     */
} pn_gemm_desc;

pn_status pn_group_create_smallm(const pn_gemm_desc *descs, int count, pn_group **out);

/* Several prefill products as one launch: the projections of a decoder layer
 * that can run together because their inputs are ready together (q, k and v;
 * gate and up), so that their tiles fill the device as one launch instead of
 * three or two that each leave part of it idle.  Each entry is one
 * pn_gemm_prefill problem (arguments, checks and results as there; M may
 * differ between entries); the entries may mix types and shapes.  At most
 * PN_PREFILL_GROUP_MAX entries, else PN_EINVAL; the first entry that fails a
 * check gives the status and nothing is enqueued.  Allocates nothing (the
 * entries travel in the launch's arguments); enqueued on `stream`. */
#define PN_PREFILL_GROUP_MAX 8
pn_status pn_gemm_prefill_group(const pn_gemm_desc *descs, int count, void *stream);

/* Enqueue all problems of a plan (either kind) as one launch on `stream`
 * (plus the rotation launch ahead of it for PN_DESC_ROTATE entries).  Runs
 * of one plan must be ordered (one stream, or waits between streams): a run
 * resets the plan's tile counters as its last wave finishes, ready for the
 * next run.  PN_EUNSUPPORTED if the device current at this call is not the
 * plan's. */
pn_status pn_group_run(const pn_group *g, void *stream);

/* Free a plan (NULL is allowed).  Synchronises the device first. */
void pn_group_destroy(pn_group *g);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, serving loops or harnesses that forbid hipMalloc): the problems of
 * a pn_group_create plan, run at once without a plan.  Results are those of
 * pn_group_create + pn_group_run on the same descriptors (the same kernel
 * choice and tile order; no PN_DESC_ROTATE entries).
 *
 * The plan (problem table, tile order, tile-pool counters) is written into a
 * library-owned device buffer of PN_BATCH_BYTES by one small kernel ahead of
 * the GEMV launch, both on `stream`; the buffer is a static device array, one
 * per GPU, held until the process ends.  The call allocates nothing and takes
 * the descriptors (a host array) by value.  Every call on a GPU shares that
 * GPU's buffer: calls on one stream are ordered, but calls that overlap on
 * one GPU (two streams, or other host threads) race and must not be made.
 *   count : 1..PN_BATCH_MAX_PROBLEMS, else PN_EINVAL (< 1) or
 *           PN_EUNSUPPORTED (too many)
 *   rows  : on the row-tile kernel at most PN_BATCH_MAX_ROWS rows in all
 *           (16-row tiles), else PN_EUNSUPPORTED
 * Other checks and errors as pn_group_create (PN_DESC_ROTATE entries return
 * PN_EUNSUPPORTED). */
#define PN_BATCH_MAX_PROBLEMS 32
#define PN_BATCH_MAX_ROWS (65536 * 16)
#define PN_BATCH_BYTES (17 * 4096 + 4096 + 4 * 65536)
pn_status pn_gemv_batch(const pn_gemv_desc *descs, int count, void *stream);

/* Streaming-read probe: the practical HBM read ceiling of the device,
 * measured in the same harness as the GEMV (the v100-skinny README, "Kernel
 * benchmarks", rates its kernels against a measured read-only ceiling).  One
 * launch reads `*bytes_read` bytes (the largest multiple of the launch's
 * granule, 1 KiB per wave, not above `bytes`) from `buf` with
 * 16-byte nontemporal DMA loads into LDS (each wave a contiguous share) and
 * writes a checksum word per lane to `scratch`.
 *   buf     : device, 16-byte aligned, `bytes` readable
 *   scratch : device, 4-byte aligned, pn_read_probe_scratch_bytes() bytes
 * Returns PN_ESHAPE if `bytes` is too small or `scratch_bytes` too small. */
size_t pn_read_probe_scratch_bytes(void);
pn_status pn_read_probe(const void *buf, size_t bytes, void *scratch, size_t scratch_bytes,
                        size_t *bytes_read, void *stream);

/* ---------------------------------------------------------------------------
 * The attention side of a decoding step: what runs between a layer's packed
 * products (q, k, v in; o out) and after the head, over a paged cache that
 * holds keys and values in pn4t blocks.
 *
 * One step: pn_kv4_plan turns request lengths into slots, positions and block
 * tables; in every layer pn_kv4_store norms and rotates the queries and keys
 * the products gave and quantizes keys and values into the cache, and
 * pn_kv4_attn attends over it; pn_spec_verify accepts or replaces drafted
 * tokens.  None of them allocates, waits or reads device data on the host,
 * and all can be captured into a HIP graph.
 *
 * Values read from device memory (lengths, tables, slots, tokens) cannot be
 * checked on the host.  The kernels bound every one of them: a bad page or
 * slot is left out, never followed.
 *
 * The cache.  A page holds page_size tokens of every key-value head; element
 * blocks of PN_KV4_BLOCK = 64 along a head are pn4t blocks (a signed fp16
 * scale d and 64 four-bit codes n, value d * (n - 8), packed as in a pn4t
 * word), with codes and scales held apart so that every load is aligned.
 * Pages follow each other; in a page, heads follow each other; a head has,
 * for token o of the page and R = dim / 64 blocks:
 *   K codes   page_size * dim / 2 bytes: row o of dim / 8 words, natural word
 *             8 b + 4 h + g (b < R, h < 2, g < 4) at place g * 2 R + 2 b + h
 *   V codes   page_size * dim / 2 bytes: word w of token o at 4-byte place
 *             ((o / 4) * (dim / 8) + w) * 4 + o % 4
 *   K scales  page_size * R fp16: token o, block b at o * R + b
 *   V scales  likewise
 * Keys are stored normed and rotated.  Slot s is token s % page_size of page
 * s / page_size.  Calls refuse (PN_EUNSUPPORTED) caches of more than 65535
 * heads or whose page has 2^31 bytes or more. */
#define PN_KV4_BLOCK 64
typedef struct pn_kv4_cache {
    void *pages;       /* device, 16-byte aligned, num_pages * pn_kv4_page_bytes */
    int32_t num_pages; /* >= 1                                                   */
    int32_t page_size; /* tokens: 16, 32, 64, 128 or 256                         */
    int32_t heads;     /* key-value heads, >= 1                                  */
    int32_t dim;       /* elements of a head: 64, 128 or 256                     */
} pn_kv4_cache;

/* Bytes of one page; 0 for a page size or dim outside the list, or heads < 1. */
size_t pn_kv4_page_bytes(int page_size, int heads, int dim);

/* Block tables, slots and positions of one step, from request lengths, on the
 * device and in one launch.  Request i has ctx_len[i] tokens in the cache,
 * brings new_len[i] more (either may be 0; negative reads as 0) and holds
 * held[i] pages: entries 0 .. held[i] - 1 of its table row.  For i < B:
 *   need     = ceil((ctx_len + new_len) / page_size)
 *   table[i][held .. need-1] = the next need - held entries of free_pages
 *            (requests in order; -1 once they are used up); other entries of
 *            the row are neither read nor written (those below held are read)
 *   held_out = max(held, need),   kv_len = ctx_len + new_len
 *   q_start  = sum of new_len over earlier requests (B + 1 entries)
 * and for the step's tokens in order, t < max_tokens:
 *   positions[t] = ctx_len[i] + its place in the request, -1 past the last
 *   slots[t]     = page * page_size + position % page_size, -1 where the
 *                  token has no page
 *   info[0] = entries of free_pages taken (<= num_free)
 *   info[1] = tokens without a place: past the free pages, past max_pages
 *             columns or past max_tokens, or in a column whose entry (held or
 *             fresh) is negative
 * A request keeps pages that rejected drafts left ahead of its tokens, so a
 * caller lowers ctx_len freely and returns pages only when a request ends.
 * Columns from max_pages on take fresh pages like the others (info[0], and the
 * requests behind get later ones) though no entry keeps them, so a caller holds
 * ctx_len + new_len within max_pages * page_size.
 * held_out counts the columns of -1 that a shortage left, too, and columns that
 * are held are not filled again.  To bring lost tokens again, a caller passes
 * as held the entries before the row's first -1, and as ctx_len at most their
 * tokens.
 *   table    : int32, B rows of ld_table >= max_pages; page ids
 *   outputs  : (table among them) must not overlap each other or an input,
 *              so kv_len is not ctx_len and held_out is not held
 *   B        : 1 .. PN_KV4_MAX_BATCH;  num_free >= 0;  max_tokens >= 1
 * Sums saturate at INT32_MAX. */
#define PN_KV4_MAX_BATCH 8192
pn_status pn_kv4_plan(const int32_t *ctx_len, const int32_t *new_len, const int32_t *held, int B,
                      const int32_t *free_pages, int num_free, int page_size, int32_t *table, int64_t ld_table,
                      int max_pages, int32_t *held_out, int32_t *q_start, int32_t *kv_len, int32_t *positions,
                      int64_t *slots, int64_t max_tokens, int32_t *info, void *stream);

/* Queries, keys and values of T tokens on their way from a layer's products:
 * for each token t and each head of q and k
 *   y  = x * g / sqrt(mean(x^2) + eps)            (gain NULL: y = x)
 *   (a, b) -> (a cos - b sin, a sin + b cos)       over rot / 2 pairs, with
 *             angle positions[t] * inv_freq[i] for pair i: elements (i,
 *             i + rot/2), or (2 i, 2 i + 1) with pairs != 0; elements from
 *             rot on stay
 * Queries are rounded to fp16 into q_out; keys, and values as they come, are
 * quantized into the cache at slots[t].  The block rule is the weights': d =
 * fp16_rne(-w / 8) with w the element of largest magnitude (the lowest index
 * of equals), code = 8 + clamp(rint(y / d), -8, 7), ties to even; d = 0 gives
 * code 8; |d| saturates at 65504; a NaN is stored as 0.  Keys are computed
 * and both are quantized in fp64, so codes do not depend on the order of
 * sums; queries in fp32, angles in fp64.
 * A token with a negative position is skipped, one with a slot outside the
 * cache is not stored (its query is written).  Slots must differ.
 *   q, k, v   : T rows of q_heads (or the cache's heads) * dim elements, fp32
 *               or fp16 (PN_ROWS_*), 16-byte aligned, ld in elements, >= the
 *               row and a multiple of 8 (fp16) or 4 (fp32).  q NULL: keys
 *               and values only; k and v both NULL: queries only
 *   q_out     : fp16, T rows, 16-byte aligned, ldo >= q_heads * dim and a
 *               multiple of 8; must not overlap q
 *   rot       : 0 .. dim, a multiple of 16 (else PN_EUNSUPPORTED); inv_freq
 *               rot / 2 fp32 values, NULL only with rot = 0
 *   T         : >= 0 (0 does nothing) */
enum { PN_ROWS_F32 = 0, PN_ROWS_F16 = 1 };
typedef struct pn_kv4_store_desc {
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv;
    const float *q_gain, *k_gain; /* fp32 [dim], 16-byte aligned, or NULL */
    const float *inv_freq;
    const int32_t *positions;     /* [T] */
    const int64_t *slots;         /* [T], 8-byte aligned; may be NULL without k, v */
    uint16_t *q_out;
    int64_t ldo;
    int64_t T;
    int32_t row_type;             /* PN_ROWS_F32 or PN_ROWS_F16, of q, k and v */
    int32_t q_heads;
    int32_t rot;
    int32_t pairs;
    float eps;
} pn_kv4_store_desc;
pn_status pn_kv4_store(const pn_kv4_cache *cache, const pn_kv4_store_desc *d, void *stream);

/* The cached keys and values of T slots as fp32, d * (n - 8) exactly: k[t] and
 * v[t] rows of heads * dim, 16-byte aligned (either may be NULL); a slot
 * outside the cache gives zeros.  The check path of pn_kv4_store, and how a
 * request's cache is read back.  T * heads * dim / 8 <= 2^32 - 256, else
 * PN_EUNSUPPORTED. */
pn_status pn_kv4_load(const pn_kv4_cache *cache, const int64_t *slots, int64_t T, float *k, float *v, void *stream);

/* Attention of a ragged batch over the cache.  Request i has queries
 * q_start[i] .. q_start[i+1]-1, the last of its kv_len[i] tokens: query j of
 * Q stands at position p = kv_len - Q + j.  Query head h reads key-value head
 * h / (q_heads / heads).
 *   out = sum_t w_t v_t / sum_t w_t,   w_t = exp(scale * q . k_t)
 * over the visible tokens t <= p; with window > 0 only t > p - window or
 * t < sinks.  A token whose table entry is not a page of the cache is not
 * visible; a query that sees nothing gives zeros.  Masked places may hold any
 * bytes.
 * Scores (from exact codes) and sums are fp32; weights and values are rounded
 * once each to fp16.
 *   q, out   : fp16, total_q rows, 16-byte aligned, ld >= q_heads * dim and a
 *              multiple of 8; must not overlap
 *   table    : int32, B rows of ld_table >= ceil(max_kv / page_size)
 *   scale    : finite, up to 2^70; scale * q . k_t below 2^24
 *   max_q    : at least every request's queries (those past it are left out)
 *   max_kv   : at least every kv_len (keys past it are left out)
 *   sinks    : >= 0, read only with window > 0 (0: no window)
 *   ws       : device, 16-byte aligned, ws_bytes (may be NULL with 0): room
 *              for the parts of rows whose keys are split over workgroups.
 *              Any size is right; pn_kv4_attn_workspace says how much the
 *              call can use (less means fewer splits).  One workspace serves
 *              calls that follow each other on a stream; calls that may
 *              overlap need their own.
 * PN_EUNSUPPORTED: B or q_heads > 65535, total_q or max_kv > 2^30 - 1, or max_q
 * * q_heads / heads > 2^29 - 1. */
size_t pn_kv4_attn_workspace(const pn_kv4_cache *cache, int q_heads, int B, int64_t total_q, int64_t max_q,
                             int64_t max_kv, int window, int sinks);
pn_status pn_kv4_attn(const pn_kv4_cache *cache, const uint16_t *q, int64_t ldq, int q_heads, const int32_t *q_start,
                      const int32_t *kv_len, const int32_t *table, int64_t ld_table, int B, int64_t total_q,
                      int64_t max_q, int64_t max_kv, float scale, int window, int sinks, uint16_t *out, int64_t ldo,
                      void *ws, size_t ws_bytes, void *stream);

/* The same for requests that share a long prefix (a system prompt, a document):
 * its keys and values are read and multiplied once for all of a group's
 * queries, and joined with each request's own.  Group g is requests g_start[g]
 * .. g_start[g+1] - 1, whose first shared[g] pages are prefix[g][0 ..
 * shared[g] - 1]; requests outside of all groups have no prefix.
 *   out as pn_kv4_attn (window 0), over the tokens t <= p: those below
 *   shared[g] * page_size from the pages in prefix[g], the others from the
 *   pages in the request's own row of table, at their own columns
 * Columns below shared[g] of a table row are not read, unless a query of the
 * request stands inside the shared pages: then all of that request's pages are
 * its own row's (as pn_kv4_plan's rows hold them).  A prefix ends with a page;
 * tokens behind its last whole page are each request's own.  Roundings are
 * pn_kv4_attn's but for one: shared tokens' weights are summed after they are
 * rounded to fp16, which pn_kv4_attn does before.
 * A call is two launches or three, and pays where a group has many queries on a
 * long prefix: 64 behind 16384 tokens 3 times as fast as pn_kv4_attn for each,
 * 4 behind 1024 or 16 of 8 drafts behind 5024 no faster.  Work is dealt as if
 * no request had more than max_kv - max_shared * page_size tokens of its own:
 * one that has more (outside of all groups, behind a shorter prefix, with a
 * query inside the shared pages) may have a single workgroup a head and tile
 * read them (16616 tokens, 128 wide: 93 us more).  Such requests do better in a
 * call of pn_kv4_attn.
 *   g_start    : int32 [G + 1], not decreasing;  shared: int32 [G], below 1: none
 *   prefix     : int32, G rows of ld_prefix >= max_shared
 *   max_shared : >= 1, at least every shared[g] (of a larger one the first
 *                max_shared pages are shared); best the largest shared[g]
 *   other arguments as for pn_kv4_attn
 *   ws         : device, 16-byte aligned, what pn_kv4_attn_shared_workspace
 *                says (less than the call needs: PN_ESHAPE).  That grows with
 *                B, G, total_q, max_q and max_kv, so that what the largest
 *                call needs serves every smaller one.  Sums of the shared keys
 *                are kept in fp32 for all queries: 4 * total_q * q_heads * dim
 *                bytes are part of it.  Calls that may overlap need their own
 * PN_EUNSUPPORTED: as pn_kv4_attn; G > 65535, max_shared * page_size > 2^30 - 1,
 * total_q * q_heads / heads > 2^29 - 1, B * q_heads * (max_q / 16 + 1) > 2^31 - 1,
 * or a launch of 2^23 workgroups (about heads times the larger of the requests
 * and the groups, for each tile of rows). */
size_t pn_kv4_attn_shared_workspace(const pn_kv4_cache *cache, int q_heads, int B, int G, int64_t total_q,
                                    int64_t max_q, int64_t max_kv, int64_t max_shared);
pn_status pn_kv4_attn_shared(const pn_kv4_cache *cache, const uint16_t *q, int64_t ldq, int q_heads,
                             const int32_t *q_start, const int32_t *kv_len, const int32_t *table, int64_t ld_table,
                             int B, const int32_t *g_start, const int32_t *prefix, int64_t ld_prefix,
                             const int32_t *shared, int G, int64_t total_q, int64_t max_q, int64_t max_kv,
                             int64_t max_shared, float scale, uint16_t *out, int64_t ldo, void *ws, size_t ws_bytes,
                             void *stream);

/* Verification of drafted tokens against the target's probabilities, from
 * given random numbers u in [0, 1).  Request i has n = n_draft[i] drafts
 * (clamped to 0..k; NULL: k), target rows p_0 .. p_k and, with `draft`, rows
 * q_0 .. q_{k-1}:
 *   draft j is accepted if all before it were and u[i][j] * q_j(x_j) <
 *   p_j(x_j) (compared exactly; without `draft` q_j(x_j) = 1; a token outside
 *   0..V-1 is refused);
 *   with a = accepted drafts, one more token is drawn from r = max(p_a - q_a,
 *   0) if a < n (without `draft`: p_a with x_a's entry 0), else from p_n: the
 *   first index whose inclusive prefix sum (fp64) is above u[i][k] * sum r.
 * Entries of r and p_a that are not positive and finite count as 0.  If r has
 * none, the token is drawn from p_a; if that has none either it is -1.
 *   out[i]      : the accepted drafts, the drawn token, then -1 (k + 1)
 *   accepted[i] : a
 *   target  : fp32, row (i, j) at (i * (k + 1) + j) * ldt, ldt >= V
 *   draft   : fp32, row (i, j) at (i * k + j) * ldd, ldd >= V, or NULL
 *   tokens  : int32, B rows of ld_tok >= k;  u : fp32, B rows of ldu >= k + 1;
 *   out     : int32, B rows of ld_out >= k + 1
 *   B 1..65535, k 0..1024, V 1..2^31-1
 *   ws      : device, 8-byte aligned, at least pn_spec_workspace(B, V) bytes */
size_t pn_spec_workspace(int B, int64_t V);
pn_status pn_spec_verify(const float *target, int64_t ldt, const float *draft, int64_t ldd, const int32_t *tokens,
                         int64_t ld_tok, const int32_t *n_draft, const float *u, int64_t ldu, int B, int k, int64_t V,
                         int32_t *out, int64_t ld_out, int32_t *accepted, void *ws, size_t ws_bytes, void *stream);

/* Between two blocks of a decoder: the norm of what a block gave, its gate and
 * residual scale, the sum with the residual stream, and the norm ahead of the
 * next block's products, in one pass.  For each of T rows of n elements
 *   u  = y                                            (post 0)
 *        y * post_gain / sqrt(mean(y^2) + eps)        (post 1)
 *   h' = h + scale * chan_scale * g(z) * u            (y NULL: h' = h)
 *   x  = fp16(h' * pre_gain / sqrt(mean(h'^2) + eps))
 * with g(z) = 1, z, 1 / (1 + exp(-z)) or z / (1 + exp(-z)) (PN_GATE_*; both of
 * the last are 0 at z = -inf), in fp32 throughout (squares that leave its range
 * count as infinite, x is 0 then); gains and chan_scale that are NULL count as 1.  x is what
 * pn_gemv, pn_gemm_smallm and pn_gemm_prefill read.
 *   h, h_out : fp32 rows.  h_out may be h (same ld) or NULL (only x wanted)
 *   y, z     : rows of row_type (PN_ROWS_*); z with a gate only, ldz 0: one row
 *              for all
 *   x        : fp16 rows, or NULL (only h_out wanted)
 *   gains    : fp32 [n]; post_gain with post only
 *   All 16-byte aligned; ld in elements, >= n and a multiple of 4 (fp32) or 8
 *   (fp16).  Elements behind a row's n are neither read nor written.  Outputs
 *   overlap no input (but h_out = h) and not each other, else PN_EINVAL.
 *   scale finite; eps finite, >= 0;  T >= 0 (0 does nothing);
 *   n 1 .. PN_NORM_MAX (else PN_EUNSUPPORTED). */
#define PN_NORM_MAX 32768
enum { PN_GATE_NONE = 0, PN_GATE_PLAIN = 1, PN_GATE_SIGMOID = 2, PN_GATE_SILU = 3 };
typedef struct pn_residual_norm_desc {
    const float *h;
    const void *y, *z;
    const float *post_gain, *chan_scale, *pre_gain;
    float *h_out;
    uint16_t *x;
    int64_t ldh, ldy, ldz, ldho, ldx;
    int64_t T, n;
    int32_t row_type;             /* PN_ROWS_F32 or PN_ROWS_F16, of y and z */
    int32_t gate;                 /* PN_GATE_*                              */
    int32_t post;                 /* norm of y                              */
    float scale, eps;
} pn_residual_norm_desc;
pn_status pn_residual_norm(const pn_residual_norm_desc *d, void *stream);

/* Log probabilities of given tokens, entropy and the most probable
 * alternatives of rows of logits: with p = softmax(scale * x) over a row's V
 * entries
 *   logp[r][j]     = ln p(tokens[r][j]);  -inf for a token outside 0..V-1
 *   entropy[r]     = - sum p ln p
 *   top_ids[r][i], top_logp[r][i] = the K entries of largest x, largest first,
 *                    the lower index of equals, and their ln p
 * An entry of -inf (a masked one) or NaN has p = 0 and is no alternative; +inf
 * counts as the largest finite value of fp32.  Places past the alternatives there are
 * get -1 and -inf.  A row without a finite entry gives -inf, entropy 0 and no
 * alternatives.  The sum of exp is fp64, the entropy's sum fp32; results
 * are rounded once to fp32.
 *   logits   : rows of row_type (PN_ROWS_*), ld >= V elements, any alignment
 *              of its type
 *   scale    : 2^-100 .. 2^64 (the inverse of a temperature)
 *   tokens   : int32, rows of ld_tok >= n_tok; n_tok >= 0 (0: may be NULL, and
 *              logp too); logp: rows of ld_lp >= n_tok
 *   entropy  : or NULL
 *   K        : 0 .. PN_LOGPROBS_MAX_TOP (0: top_ids and top_logp may be NULL);
 *              rows of ld_top >= K
 *   rows     : >= 0 (0 does nothing);  V 1..2^31-1;  rows * ceil(V / 1024) <
 *              2^31, else PN_EUNSUPPORTED
 *   ws       : device, 8-byte aligned, at least pn_logprobs_workspace bytes,
 *              which grow with rows, V and K; calls that may overlap need
 *              their own
 *   Outputs and ws overlap neither inputs nor each other, else PN_EINVAL. */
#define PN_LOGPROBS_MAX_TOP 64
size_t pn_logprobs_workspace(int64_t rows, int64_t V, int K);
pn_status pn_logprobs(const void *logits, int row_type, int64_t ld, int64_t rows, int64_t V, float scale,
                      const int32_t *tokens, int64_t ld_tok, int n_tok, float *logp, int64_t ld_lp, float *entropy,
                      int K, int32_t *top_ids, float *top_logp, int64_t ld_top, void *ws, size_t ws_bytes,
                      void *stream);

/* Text for a status code. */
const char *pn_status_str(pn_status e);

/* Kernel variant chosen by this thread's last successful enqueue (a census
 * for benchmarks so that no fallback route goes unreported); values are
 * listed by pn_variant_name. */
int pn_last_variant(void);
const char *pn_variant_name(int v);

#ifdef __cplusplus
}
#endif
#endif
