/*
 * The drafter's cache in 8 bits: quantised as it is written, read back, and
 * attended to ("Chunk 66.0", magik.net seg_66/chunk_0: a drafter with KV
 * caching proposes the trees; its one-token attention is bound by the bytes
 * of its cache, and 8 bits halve them).
 *
 * An element of the cache is an e4m3 number c (1 sign, 4 exponent and 3
 * mantissa bits, largest 448) and stands for c * scale, with a scale for each
 * block of tokens and key head, of keys and of values.  Token t of a page lies
 * in its block t / block_tokens; a page's last block may be a short one.
 * Scales are 32-bit numbers in [DDTREE_DRAFT8_SCALE_MIN, _MAX]; the append
 * writes powers of two, so a block that moves to a larger scale keeps its
 * numbers but for those that become subnormal.
 *
 * Conventions as in ddtree_verify.h.
 */
#ifndef DDTREE_DRAFT8_H_
#define DDTREE_DRAFT8_H_

#include "ddtree_draft.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DDTREE_DRAFT8_MAX_BLOCK 4096          /* block_tokens * head_dim */
#define DDTREE_DRAFT8_SCALE_MIN 5.4210108624275222e-20f  /* 2^-64 */
#define DDTREE_DRAFT8_SCALE_MAX 7.9228162514264338e28f   /* 2^96 */

/* Element (page, token, head, column) of k and of v lies page * page_stride +
 * token * token_stride + head * head_stride + column bytes behind the pointer;
 * its scale is number (page * blocks + token / block_tokens) * n_kv_heads +
 * head of k_scale or v_scale, with blocks = ceil(page_size / block_tokens). */
typedef struct ddtree_draft8_cache {
  void* k;               /* 16-byte aligned, e4m3 codes                           */
  void* v;
  float* k_scale;        /* [n_pages, blocks, n_kv_heads], contiguous             */
  float* v_scale;
  int64_t n_pages;       /* n_pages * page_size <= 2^31 - 1                       */
  int64_t page_stride;   /* bytes, multiples of 16 below 2^36                     */
  int64_t token_stride;
  int64_t head_stride;
  int32_t page_size;     /* tokens of a page, 1 .. DDTREE_MAX_PAGE_SIZE, any number */
  int32_t n_kv_heads;    /* 1 .. DDTREE_MAX_HEADS                                 */
  int32_t head_dim;      /* 64, 128 or 256                                        */
  int32_t block_tokens;  /* 1 .. DDTREE_DRAFT8_MAX_BLOCK / head_dim, any number up to page_size */
} ddtree_draft8_cache_t;

/*
 * Queries, keys and values of n_tokens new tokens, as ddtree_draft_append, the
 * keys and values quantised:
 *   q_out[n, h]                 = R(positions[n]) norm(q[n, h], q_weight)
 *   k cache, scales [slots[n]]  = quantised R(positions[n]) norm(k[n, h], k_weight)
 *   v cache, scales [slots[n]]  = quantised v[n, h]
 * Keys are quantised from their 32-bit values.  Per key head, with m the
 * largest finite magnitude of the rows that the call writes to a block:
 *   - A block whose first token is among them starts afresh: its scale is the
 *     least power of two s with m <= 448 s (from 2^-64 to 2^96; 1 where m is
 *     0), and its other tokens hold nothing from then on.
 *   - Otherwise the block keeps its scale if m <= 448 times that; if not, it
 *     takes the one that the rows need, and the tokens that it holds already
 *     are quantised again with it.  A scale that is no number from 2^-64 to
 *     2^96 counts as none: the block starts afresh.
 * Codes are rounded to the nearest, ties to even; what lies beyond 448 becomes
 * 448 (infinities too), NaN stays NaN.
 * So a request's tokens are to be written in order, as ddtree_step_maps lays
 * them out, and in a call tokens of the same block must follow one another
 * in the list, nothing between them, no padding token either: of a block that a
 * call names in several places, or of a slot that it names twice, the contents
 * would be a mixture (of that block alone).  Tokens of rejected drafts may be
 * overwritten; their block's scale stays.
 *   dtype          DDTREE_BF16 or DDTREE_FP16, of q, k, v, weights and q_out
 *   n_tokens, n_heads, rope, strides, positions, slots, status as in
 *   ddtree_draft_append; slot = page * page_size + token in page
 * Errors: DDTREE_EINVAL, DDTREE_EUNSUPPORTED, DDTREE_ELAUNCH.
 */
DDTREE_API int ddtree_draft8_append(int64_t n_tokens, int n_heads, int dtype, const ddtree_draft8_cache_t* cache,
                                    const ddtree_rope_t* rope, const void* q, int64_t q_stride, const void* k,
                                    int64_t k_stride, const void* v, int64_t v_stride, const void* q_weight,
                                    const void* k_weight, float eps, const int32_t* positions, const int32_t* slots,
                                    void* q_out, int64_t q_out_stride, uint32_t* status, struct CUstream_st* stream);

/*
 * Rows of the cache read back: k_out[n, h] = k cache[slots[n], h] in 16 bits,
 * v_out likewise; a product is rounded once (exact in bf16 where the scale is
 * a power of two; fp16 holds less range, and what lies beyond it becomes an
 * infinity).
 *   n_rows        0 .. DDTREE_APPEND_MAX_TOKENS (0: nothing happens)
 *   slots         [n_rows] int32; -1: the row is left as it is.  Others outside
 *                 the cache: DDTREE_ST_BAD_INDEX, left as they are.  A slot may
 *                 be named any number of times.
 *   k_out, v_out  dtype, rows *_stride elements apart (multiples of 8), heads
 *                 head_dim apart; one of them may be NULL
 *   status        uint32, OR-ed (the caller clears it), or NULL.  A scale that
 *                 is no number from 2^-64 to 2^96 sets DDTREE_ST_BAD_SCALE, and
 *                 its rows are 0.
 * Errors: DDTREE_EINVAL, DDTREE_EUNSUPPORTED, DDTREE_ELAUNCH.
 */
DDTREE_API int ddtree_draft8_read(int64_t n_rows, int dtype, const ddtree_draft8_cache_t* cache, const int32_t* slots,
                                  void* k_out, int64_t k_out_stride, void* v_out, int64_t v_out_stride,
                                  uint32_t* status, struct CUstream_st* stream);

/* Fields are outputs of ddtree_draft8_attention_plan except q_stride and
 * out_stride, which the caller may set afterwards (0: contiguous tokens). */
typedef struct ddtree_draft8_plan {
  int32_t n_tokens, n_heads, n_kv_heads, head_dim, dtype, page_size, block_tokens;
  int32_t window, n_sinks;   /* window 0: no window                              */
  int32_t row_tiles;         /* work items of a key head: each 16 query heads    */
  int32_t tile_keys;         /* keys of an inner tile                            */
  int32_t n_shares;          /* CTAs, each with an equal share of all key tiles  */
  int64_t q_stride, out_stride;   /* elements between tokens, multiples of 8     */
  int64_t workspace_bytes;
} ddtree_draft8_plan_t;

/* As ddtree_draft_attention_plan; dtype: of q and out. */
DDTREE_API int ddtree_draft8_attention_plan(int n_tokens, int n_heads, const ddtree_draft8_cache_t* cache, int dtype,
                                            int window, int n_sinks, int num_sms, ddtree_draft8_plan_t* plan);

/* As ddtree_draft_attention_workspace_size. */
DDTREE_API size_t ddtree_draft8_attention_workspace_size(const ddtree_draft8_plan_t* plan);

/*
 * ddtree_draft_attention over the 8-bit cache: the same visible keys, page
 * table, outputs and data errors.  Besides, a key with a scale that is no
 * number from 2^-64 to 2^96 (of its key or its value) sets DDTREE_ST_BAD_SCALE
 * and is dropped.
 *
 * e4m3 numbers are exact in fp16, and products run there: a query row is moved
 * by a power of two so that its largest element fills fp16's range (what is
 * 2^-39 of it or less is lost), scores, maxima and sums are in 32 bits, and the
 * weight p_j vscale_j of a value row is rounded to fp16 (half a step of it,
 * 2^-11) relative to the unit's largest: a row counts down to 2^-34 of that.
 * The sums take p_j unrounded, but lose a key whose weight is below 2^-130 of the
 * largest: value scales of a request's keys are to lie within 2^100 of each
 * other.  The products cut their sums off at 32 bits, which takes some 4e-9 of
 * sum p |v| for each key: a warp's sums start anew every 8,192 keys and are added
 * up, so that this stays below 5e-5.  An output is rounded once.  Equal inputs
 * give equal bits.
 * Errors: as ddtree_draft_attention.
 */
DDTREE_API int ddtree_draft8_attention(const ddtree_draft8_plan_t* plan, const void* q,
                                       const ddtree_draft8_cache_t* cache, const int32_t* page_table, int table_rows,
                                       int table_stride, const int32_t* token_rows, const int32_t* positions,
                                       float sm_scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                       struct CUstream_st* stream);

#ifdef __cplusplus
}
#endif

#endif /* DDTREE_DRAFT8_H_ */
