/*
 * sar_ops.h -- single-kernel entry points of the hybrid step, for per-kernel
 * parity tests and for the tile-quantisation sweep.
 *
 * The GEMM is the "one GEMM per weight over all [Lp+Bd, H] rows" of
 * "SARATHI: Efficient LLM Inference by Piggybacking Decodes with Chunked
 * Prefills" (reading notes, part 2 section 3).  Its row-tile choice is what the
 * same notes' part 3 section 3 (tile quantisation: 257 rows need a third
 * 128-row block) and the Sarathi-Serve digest (section 2, Q2 item 3: 257 vs
 * 256 tokens costs +32% prefill time) are about; the variants below let a
 * caller pick the tiling and measure it.
 */
#ifndef SAR_OPS_H
#define SAR_OPS_H

#include <stdint.h>

#include "sar.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Epilogues applied to the fp32 accumulator D = A . W^T. */
enum {
  SAR_EPI_STORE = 0,    /* C [M, N] in the storage type = D                          */
  SAR_EPI_RESIDUAL = 1, /* C fp32 [M, N] = D + R (R fp32 [M, N]; R may equal C)      */
  SAR_EPI_SWIGLU = 2,   /* W is gate/up interleaved in 64-row blocks, [2F, K]; C [M, F]
                           in the storage type = silu(D_gate) * D_up                 */
  SAR_EPI_F32 = 3       /* C fp32 [M, N] = D                                         */
};

/* Tilings.  All run tcgen05 MMAs (16-bit x 16-bit -> fp32 in tensor memory) fed by
 * TMA from 128-byte-swizzled shared memory, in a persistent kernel. */
enum {
  SAR_GEMM_AUTO = 0,  /* the library's choice for (M, N, K)                        */
  SAR_GEMM_M128_N128 = 1, /* 128 token rows x 128 weight rows per tile              */
  SAR_GEMM_M128_N256 = 2, /* 128 token rows x 256 weight rows per tile              */
  SAR_GEMM_SWAP = 3,      /* weights on the MMA's M side (128 rows), tokens on its N
                             side padded to 16 (M <= 256): no 128-row quantisation */
  SAR_GEMM_M256_N128 = 4, /* 256 token rows (two 128-row MMAs sharing one weight
                             tile) x 128 weight rows per tile                        */
  SAR_GEMM_PAIR_N256 = 5, /* 256 token rows x 256 weight rows per tile over a pair of
                             CTAs (2-CTA cluster): one M = 256 MMA reads each CTA's
                             128 token rows and half of the weight rows, so each SM
                             loads half the weight tile                             */
  SAR_GEMM_PAIR_N128 = 6, /* the same with 128 weight rows per tile                 */
  SAR_GEMM_PAIR_N192 = 7, /* the same with 192 weight rows per tile (not for the
                             SwiGLU epilogue, whose gate/up blocks are 128 wide)    */
  /* Optional flag for the swap tiling with at most 128 token rows: two CTAs
   * per SM, each with half the pipeline, so twice as many weight slabs are in
   * flight per SM (the memory-bound regime). */
  SAR_GEMM_TWO_CTAS = 0x1000,
  /* Optional flag for the in-place fp32 residual epilogue (non-swap tilings):
   * stream-K.  Every resident CTA (pair) takes an equal, contiguous share of
   * all tiles' 64-wide K slabs, so a few tiles spread over all SMs instead of
   * leaving a partial wave; a share that covers part of a tile's K range adds
   * its partial sum into C atomically (as split-K does).  Each token group's
   * weight slabs are shared out separately, so the groups read a weight slab
   * at the same time (once from HBM).  AUTO does not take it. */
  SAR_GEMM_STREAM_K = 0x2000
};

/* C = epilogue(A . W^T).  A [M, K], W [N, K] in the storage type `storage`
 * (SAR_STORAGE_F16 or SAR_STORAGE_BF16; device, row-major, 16-byte aligned,
 * K a multiple of 64, N a multiple of 64, M >= 1).  For SAR_EPI_SWIGLU, N is
 * 2F (the packed rows) and C has F columns.  Returns SAR_ERR_UNSUPPORTED for
 * shapes a variant cannot take. */
int sar_op_gemm(const void* a, const void* w, void* c, const void* residual, int32_t M, int32_t N,
                int32_t K, int32_t epilogue, int32_t variant, int32_t storage, void* stream);

/* Device-side status of the single-kernel entry points (sar_op_gemm,
 * sar_op_wait_check) on the current device.  Their kernels record the first
 * failure -- a bounded wait that gave up (SAR_ERR_TIMEOUT) or an index out of
 * bounds (SAR_ERR_BOUNDS) -- in one record per device instead of trapping.
 * This call synchronises the device, reads the record, clears it and returns
 * its code (SAR_OK if none); sar_last_error() then names the kernel site and
 * a detail.  The record is shared by every stream and thread on the device. */
int sar_op_sync_status(void);

/* Exercises the bounded wait that every pipelined kernel uses (no counterpart
 * in the pages; the bound keeps a stuck pipeline from holding the GPU).  One
 * thread initialises a shared-memory barrier that needs two arrivals, arrives
 * `arrivals` times (0..2) and waits for it with a limit of limit_ns
 * nanoseconds (> 0).  With two arrivals the wait completes; with fewer it
 * runs out after about limit_ns, the kernel records SAR_ERR_TIMEOUT for
 * sar_op_sync_status() and returns, and the context stays usable.  Async on
 * `stream`. */
int sar_op_wait_check(int64_t limit_ns, int32_t arrivals, void* stream);

/* y = x * rsqrt(mean(x^2) + eps) * gain per row: x fp32 [rows, hidden] (the
 * residual stream), gain fp32 [hidden], y [rows, hidden] in `storage`. */
int sar_op_rmsnorm(const void* x, const void* gain, void* y, int32_t rows, int32_t hidden,
                   float eps, int32_t storage, void* stream);

/* ---- 4-bit rows --------------------------------------------------------- */

/* Microscaled 4-bit floating point (no counterpart in the pages, which serve
 * 16-bit weights): a matrix [rows, cols] is kept as e2m1 codes q (0, 0.5, 1,
 * 1.5, 2, 3, 4, 6 with a sign) with one scale s per block of columns of a row,
 * and stands for q * s * tensor_scale.
 *   SAR_FP4_NV  blocks of 16, s an e4m3 number (sign bit clear)
 *   SAR_FP4_MX  blocks of 32, s = 2^(byte - 127); byte 255 is NaN
 * cols is a multiple of 32.
 *   codes   uint8 [rows][cols / 2], contiguous, 16-byte aligned: column 2i in
 *           byte i's low four bits (bit 3 the sign), column 2i + 1 in its high ones
 *   scales  uint8, 16-byte aligned, sar_op_fp4_scale_bytes() long.  Tiles of 128
 *           rows x 4 blocks hold 512 bytes: row r and block b of the tile at
 *           (r % 32) * 16 + (r / 32) * 4 + b.  The tiles of 128 rows follow one
 *           another along the columns (the last one padded to 4 blocks), then
 *           come those of the next 128 rows.  This is the order the product's
 *           tensor cores take them in.  Padding blocks hold zero; the bytes of
 *           rows behind the last are neither written nor used. */
enum { SAR_FP4_NV = 0, SAR_FP4_MX = 1 };

/* Length of a matrix's scales in bytes. */
int sar_op_fp4_scale_bytes(int32_t rows, int32_t cols, int32_t format, int64_t* out);

/* codes, scales = x: x device rows of `type`, row r at x + r * ldx elements
 * (ldx >= cols; any alignment of the element, 16 bytes are faster).  With
 * t = x * (1 / tensor_scale) in fp32 and a = max |t| over a block,
 *   NV  s = a / 6 rounded to e4m3 (at most 448);    q = t / s rounded to e2m1
 *   MX  s = 2^(floor(log2 a) - 2), at least 2^-127;  q = t / s rounded to e2m1
 * to nearest even, q at most 6 in magnitude; a block whose scale rounds to zero
 * is zero.  A block that holds a NaN or an infinity (in t) gets a NaN scale and
 * zero codes.  tensor_scale > 0, finite, with a finite inverse.  rows = 0 does
 * nothing; rows * cols / 16 (cols padded to whole scale tiles) stays below 2^31.
 * Async on `stream`. */
int sar_op_fp4_quantize(const void* x, int64_t ldx, int32_t rows, int32_t cols, int32_t type, int32_t format,
                        float tensor_scale, void* codes, void* scales, void* stream);

/* y = the rows that codes and scales stand for: q * s (exact) * tensor_scale in
 * fp32, rounded to `type`.  y rows as x above, below 2^31 times 16 bytes in all.
 * Async on `stream`. */
int sar_op_fp4_dequantize(const void* codes, const void* scales, int32_t rows, int32_t cols, int32_t format,
                          float tensor_scale, void* y, int64_t ldy, int32_t type, void* stream);

/* Tilings of the 4-bit product. */
enum {
  SAR_FP4_GEMM_AUTO = 0,  /* the library's choice for (M, N, K)                        */
  SAR_FP4_GEMM_SPLIT = 1, /* 128 weight rows x up to 128 token rows per tile, the K
                             range cut over a cluster's CTAs: | (count << 8) for that
                             many ranges (up to 8, one per 256 columns; else one); up
                             to 65535 tiles of either side's rows                     */
  SAR_FP4_GEMM_PAIR = 2,  /* 256 weight rows x up to 256 token rows per tile over a
                             pair of CTAs (2-CTA cluster), persistent; | (2 << 8) for
                             two K ranges per tile, a pair each                     */
  SAR_FP4_GEMM_TOKENS64 = 0x1000 /* flag for SPLIT: tiles of 64 token rows             */
};

/* C = epilogue(alpha * A . W^T) of 4-bit rows of one format: A [M, K] and W [N, K]
 * as codes and scales laid out as above, each without its tensor scale (alpha
 * holds their product).  K a multiple of 32, any M >= 0 and N >= 1,
 * each at most 2^30.
 *   SAR_EPI_STORE     C [M, N] in the 16-bit type `storage`
 *   SAR_EPI_RESIDUAL  C fp32 [M, N] = alpha * A . W^T + R (R may equal C)
 *   SAR_EPI_SWIGLU    W's rows gate/up interleaved in 64-row blocks (N a multiple
 *                     of 128); C [M, N / 2] = silu(gate) * up in `storage`
 *   SAR_EPI_F32       C fp32 [M, N]
 * C and R are contiguous; N a multiple of 4 and 16-byte aligned rows are faster.
 * Sums are fp32 as the tensor cores form them: where one does not fit 24 bits they
 * cut it off instead of rounding it, which costs up to 2^-23 of the products'
 * magnitudes per 64 columns; K ranges are then added in fp32.  The result does not
 * depend on timing.  Async on `stream`; device-side failures are read with
 * sar_op_sync_status(). */
int sar_op_gemm_fp4(const void* a, const void* a_scales, const void* w, const void* w_scales, void* c,
                    const void* residual, int32_t M, int32_t N, int32_t K, float alpha, int32_t epilogue, int32_t format,
                    int32_t variant, int32_t storage, void* stream);

/* ---- KV cache in 8 bits ------------------------------------------------- */

/* A paged cache of one layer whose keys and values are held in 8 bits (no
 * counterpart in the pages, whose cache is 16-bit): e4m3 codes q with one scale s
 * for each page and head, standing for q * s.  Half the bytes of the 16-bit pages,
 * and as much less to read for every decode.
 *   k_codes, v_codes    uint8 [num_pages][n_kv_heads][page_size][head_dim],
 *                       contiguous, 16-byte aligned
 *   k_scales, v_scales  fp32 [num_pages][n_kv_heads]
 * page_size is 16, 32 or 64, head_dim 64 or 128; num_pages * n_kv_heads *
 * page_size stays below 2^31. */
typedef struct sar_kv8 {
  void* k_codes;
  void* v_codes;
  float* k_scales;
  float* v_scales;
  int32_t num_pages, n_kv_heads, page_size, head_dim;
} sar_kv8;

/* Block tables and slot maps from request lengths, on the device, so that a
 * captured step can go from one batch to the next without the host.  Request i
 * (i < n) has lens[i] tokens in its first ceil(lens[i] / page_size) pages and
 *   new_lens[i] > 0   gets room for that many more: pages taken from the end of the
 *                     free list, request by request, into its block table
 *   new_lens[i] == 0  waits: nothing changes
 *   new_lens[i] == -1 has ended: its pages go to the end of the free list (request
 *                     by request, in table order) before any are taken
 * Results:
 *   lens_out[i]      lens[i] + new_lens[i]; 0 for a request that has ended
 *   row_offsets      [n + 1]: request i's rows are row_offsets[i] .. row_offsets[i + 1]
 *   positions, slots [max_rows]: each row's position in its request, and its place
 *                    in the cache, page * page_size + offset; rows behind the last
 *                    request's have slot -1 and position 0
 *   free_count_out   pages on the list afterwards
 * Pages go first come, first served: where a request's are not there, neither it nor
 * a request behind it that needs pages gets any; nor does a request whose rows do
 * not fit max_rows.  Such a request keeps its length and its rows' slots are -1.
 * sar_op_sync_status() reports it (SAR_ERR_NO_PAGES, or SAR_ERR_BOUNDS for the rows).
 * Also SAR_ERR_BOUNDS: a request whose length is negative (it counts as 0) or passes
 * its block table, with the new tokens too, or whose new_lens is below -1, waits; a
 * page out of range goes where it would, but rows in it have slot -1.
 * lens_out may be lens, free_count_out free_count; else no two arrays overlap.  bt_cols
 * is at most bt_stride, so that block_tables may be columns of a wider table.
 * n is at most 8192, n * bt_stride and max_rows at most 2^30.  Async on `stream`;
 * no workspace. */
typedef struct sar_page_map_args {
  const int32_t* lens;     /* [n] */
  const int32_t* new_lens; /* [n] */
  int32_t* lens_out;       /* [n] */
  int32_t* block_tables;   /* [n][bt_stride], of which bt_cols are read and written */
  int32_t* free_pages;     /* [num_pages], the first *free_count are free */
  const int32_t* free_count;
  int32_t* free_count_out;
  int32_t* row_offsets; /* [n + 1] */
  int32_t* positions;   /* [max_rows] */
  int32_t* slots;       /* [max_rows] */
  int32_t n, bt_stride, page_size, num_pages, max_rows;
  int32_t bt_cols; /* pages that a request's row of block_tables has room for; 0: bt_stride */
} sar_page_map_args;
int sar_page_map(const sar_page_map_args* args, void* stream);

/* A step's query, key and value rows behind their projection.  For every head h of
 * q and k, in fp32:
 *   norm      h = h * rsqrt(mean(h^2) + eps) * gain   (q_gain, k_gain fp32
 *             [head_dim]; NULL: none)
 *   rotation  the pair (h[i], h[i + head_dim / 2]) turned by position *
 *             rope_base^(-2 i / head_dim), the angle reduced exactly (positions
 *             NULL: none)
 * q_out and k_out (NULL: not written) get them rounded once.  With a cache, k and
 * v are also written into it at their rows' slots (from sar_page_map; a slot of -1 is
 * passed over, one out of range passed over and reported): for each page and head
 * that gets rows, a = the largest finite magnitude among them,
 *   s = the smallest power of two in [2^-40, 2^60] with a <= 448 s
 * or the page's present scale where its first new row is not the page's first and
 * that is larger; codes are h / s rounded to nearest even, at most 448 in magnitude;
 * infinities and NaN become NaN.  Where a page's scale grows, the rows in front of
 * its first new one are rounded anew under it.  A page's rows follow one another
 * in the call, with consecutive slots (otherwise that page's contents are
 * unspecified), as sar_page_map gives them.
 * Rows are `type` (SAR_TYPE_*), row r at q + r * ldq elements; q_out and k_out have
 * the 16-bit type `out_type`, which is `type` where that is 16 bits.  n_kv_heads of k
 * and v.  q may be NULL (no query heads).  16-bit rows may be written over (q_out is q,
 * of the same stride; without a cache k_out is k), else outputs overlap nothing.  16-byte
 * aligned rows are faster.  Async on `stream`. */
typedef struct sar_qk_rows {
  const void* q;
  const void* k;
  const void* v; /* with a cache */
  void* q_out;
  void* k_out;
  int64_t ldq, ldk, ldv, ldq_out, ldk_out;
  const float* q_gain;
  const float* k_gain;
  const int32_t* positions; /* [rows] */
  const int32_t* slots;     /* [rows], with a cache */
  int32_t rows, n_q_heads, n_kv_heads, head_dim, type, out_type;
  float eps, rope_base;
} sar_qk_rows;
int sar_qk_norm_rope(const sar_qk_rows* rows, const sar_kv8* cache, void* stream);

/* Attention over an 8-bit cache.  Sequence i (i < n) has lens[i] tokens in its block
 * table's pages; its rows row_offsets[i] .. row_offsets[i + 1] of q are its last
 * tokens, so row j of r stands at position p = lens[i] - r + j and sees the keys at
 * positions (p - window, p] (window 0: [0, p]).  For each head, in fp32,
 *   out = sum_k softmax_k(scale * q . K_k) V_k
 * with query head h reading KV head h / (n_q_heads / n_kv_heads).  A row that sees
 * nothing (p < 0) is zero; keys that it does not see do not touch it, whatever they
 * hold.  Single tokens and chunks may stand side by side in a call.  Codes are
 * multiplied as they are, sums are fp32; a query's elements are off by 2^-17 of the
 * largest of their row and head at most, a key's probability by 2^-11 of itself or 2^-24 of
 * its row's largest, whatever value scales lie beside one another (chunks of several rows
 * take pages slowly whose scale is more than 2^4 from most others' of their sequence).
 * Rows are 16-bit, row r at q + r * ldq elements, heads of head_dim adjacent; out
 * likewise.  max_rows bounds a sequence's rows (1: single tokens alone); max_len
 * (0: unknown) is about the longest length and only guides how work is shared
 * out.  scale 0 is 1 / sqrt(head_dim).  A cache's scales are positive and lie
 * within [2^-40, 2^60].  At most 8 query heads per KV head, 2^27 rows, 2^30 sequences and block
 * tables of 2^31 - 257 tokens.  q and out do not overlap; no row is two sequences'.
 * The workspace (device, 16-byte aligned, sar_kv8_attention_workspace() bytes; it
 * holds nothing between calls) belongs to one call at a time.
 * Sequences whose offsets are out of range or fall, whose rows pass max_rows or
 * whose length passes its block table's bt_cols pages are left out, and keys of pages out of range
 * are passed over (a row that sees no others is NaN); sar_op_sync_status() reports either.
 * Rows of no sequence stay as they are.  Async on `stream`; allocates nothing. */
typedef struct sar_kv8_batch {
  const void* q;
  void* out;
  int64_t ldq, ldo;
  const int32_t* row_offsets;  /* [n + 1] */
  const int32_t* lens;         /* [n] */
  const int32_t* block_tables; /* [n][bt_stride], of which bt_cols are read */
  void* workspace;
  int64_t workspace_bytes;
  int32_t rows, n, n_q_heads, bt_stride, storage, max_rows, max_len, window;
  float scale;
  int32_t bt_cols; /* columns of a block table, at most bt_stride; 0: bt_stride */
} sar_kv8_batch;
/* Bytes of workspace for such a call (rows, n, n_q_heads, max_rows and max_len of
 * the batch are read) on the current device. */
int sar_kv8_attention_workspace(const sar_kv8_batch* batch, const sar_kv8* cache, int64_t* bytes);
int sar_kv8_attention(const sar_kv8_batch* batch, const sar_kv8* cache, void* stream);

/* Device address of a step workspace buffer, valid until sar_model_destroy;
 * after a step on a one-layer model it holds that layer's intermediates.
 *   0: normed rows     [max_tokens, hidden] (storage type)
 *   1: rotary table    fp32, (cos, sin) of each row's position times theta_i:
 *                      for row r and frequency i, at float index
 *                      4 * ((i / 2) * max_tokens + r) + 2 * (i % 2) (frequency
 *                      pairs major, so a warp's 32 rows read 512 contiguous bytes)
 *   2: attention rows  [max_tokens, n_q_heads * head_dim] (storage type)
 *   3: SwiGLU rows     [max_tokens, ffn] (storage type)
 *   4: residual stream fp32 [max_tokens, hidden] (when the step had no hidden_out)
 *   5: q|k|v rows      fp32 [max_tokens, (n_q_heads + 2 n_kv_heads) * head_dim]
 *                      (the projection with q and k rotated; k and v are
 *                      also in the pages, rounded to the storage type; for
 *                      head_dim 128 and more than 32 rows -- a QKV projection
 *                      on 128-row token tiles -- only q is kept in fp32; the
 *                      attention kernels read k and v from the pages) */
int sar_model_debug_buffer(sar_model* m, int32_t which, void** out);

/* The step planner on the host alone (no GPU, no model): plans batch `b` as
 * sar_step would for a model of `dims` (with chunk_split as set by
 * sar_model_set_chunk_split), a cache of num_pages pages of page_size tokens
 * and a device of `sms` SMs (sar_step plans for the current device's), with
 * the same validation and errors.  layout (int32[25])
 * receives M, Lp, Bd, R, decode work items, decode partials, chunk tiles,
 * rows per chunk tile, then the offsets (int32 elements) of the metadata
 * block's arrays -- row positions, row page slots, chunk block tables,
 * decode key counts, decode block-table offsets, decode block-table lengths,
 * first partial, partial count, work items [4 each: decode, first key, end
 * key, partial or -1], decode block tables, logits rows, chunk tiles [8 each:
 * first batch row, first position, rows, block-table offset, block-table
 * length, first and end 128-key block, key-range partial slot or -1] -- its
 * total length, then the chunk key-range merges, their partial slots and the
 * merges' offset [4 each: first batch row, rows, first slot, slots], then 1
 * when the chunk tiles are listed in pairs (entries 2i and 2i + 1: two query
 * tiles of one chunk, the second possibly of 0 rows, one CTA per pair and
 * head), else 0.  The
 * block itself (what the step ships to the device) is copied to meta
 * (int32[meta_cap], may be NULL) and its length to *meta_n. */
int sar_plan_inspect(const sar_dims* dims, int32_t page_size, int32_t num_pages, int32_t sms,
                     int32_t chunk_split, const sar_batch* b, int32_t* layout, int32_t* meta, int64_t meta_cap,
                     int64_t* meta_n);

#ifdef __cplusplus
}
#endif

#endif /* SAR_OPS_H */
