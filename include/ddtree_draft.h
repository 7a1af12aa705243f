/*
 * The drafter's attention: one new token per request over its paged key and
 * value cache ("Chunk 66.0", magik.net seg_66/chunk_0: a drafter with
 * sliding-window attention and KV caching proposes the trees).
 *
 * Token n stands at position p = positions[n] of the request whose pages are
 * row token_rows[n] of the page table.  It sees itself, the window before it
 * and the first tokens of the request:
 *     K(n) = { j <= p :  j > p - window  or  j < n_sinks }   (window 0: all j <= p)
 *     out[n, h] = sum_j softmax_j(sm_scale <q[n, h], k_j>) v_j,
 *     lse[n, h] = ln sum_j exp(sm_scale <q[n, h], k_j>)
 * with the key head h / (n_heads / n_kv_heads).  Several tokens may name the
 * same row (the tokens a step has just committed, at their own positions).
 * Table entries of pages that no visible key lies in are never read, so pages
 * behind the window may have been released.
 *
 * Scores, the softmax's maxima and sums and the products' sums are held in 32
 * bits.  A probability is rounded to the cache's type (half a step of it) where
 * it meets V, as in the verify kernels, while the sums take it unrounded; fp16
 * probabilities carry a factor of 2^10 there, so that keys down to 2^-34 of the
 * largest count.  An output is rounded once.
 *
 * The work is split over the tokens' lengths in equal shares for the SMs, read
 * on the device: a plan depends on no length, and a captured call replays with
 * any.  Partial results are joined in a fixed order: equal inputs give equal
 * bits.
 *
 * Conventions as in ddtree_verify.h.
 */
#ifndef DDTREE_DRAFT_H_
#define DDTREE_DRAFT_H_

#include "ddtree_append.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DDTREE_DRAFT_MAX_TOKENS 4096
#define DDTREE_DRAFT_MAX_GROUP 64     /* query heads of one key head */

/* Fields are outputs of ddtree_draft_attention_plan except wait_limit_us,
 * q_stride and out_stride, which the caller may set afterwards (0: 2 s,
 * contiguous tokens). */
typedef struct ddtree_draft_plan {
  int32_t n_tokens, n_heads, n_kv_heads, head_dim, dtype, page_size;
  int32_t window, n_sinks;   /* window 0: no window                              */
  int32_t row_tile;          /* query rows of a work item: 16, 32 or 64          */
  int32_t tile_keys;         /* keys of an inner tile                            */
  int32_t n_shares;          /* CTAs, each with an equal share of all key tiles  */
  int32_t wait_limit_us;     /* bound of each wait inside the kernel of wide groups
                                (row_tile 64), in microseconds; one that expires sets
                                DDTREE_ST_TIMEOUT, and the call ends without it (e.g.
                                to test that path)                              */
  int64_t q_stride, out_stride;   /* elements between tokens, multiples of 8     */
  int64_t workspace_bytes;
} ddtree_draft_plan_t;

/*
 * n_tokens 1 .. DDTREE_DRAFT_MAX_TOKENS; n_heads a multiple of the cache's key
 * heads, at most DDTREE_DRAFT_MAX_GROUP times; window 0 .. 2^31-1; n_sinks
 * 0 .. 2^31-1 (without a window every key is visible anyway).
 * num_sms: 0 asks the current device, > 0 plans for that many without one.
 * Errors: DDTREE_EINVAL, DDTREE_EUNSUPPORTED (num_sms 0 and no device).
 */
DDTREE_API int ddtree_draft_attention_plan(int n_tokens, int n_heads, const ddtree_draft_cache_t* cache, int window,
                                           int n_sinks, int num_sms, ddtree_draft_plan_t* plan);

/* Workspace bytes for a plan (a multiple of 256; 256-byte aligned buffer): the
 * 256-byte status block (read with ddtree_verify_mla_check), then the shares'
 * partial results.  It keeps nothing between calls; calls that may overlap on
 * the GPU need a workspace each.  0 for a null plan. */
DDTREE_API size_t ddtree_draft_attention_workspace_size(const ddtree_draft_plan_t* plan);

/*
 *   q           [n_tokens, n_heads, head_dim] dtype, tokens plan->q_stride apart
 *   page_table  [table_rows, table_stride] int32
 *   token_rows  [n_tokens] int32, or NULL (row n)
 *   positions   [n_tokens] int32; -1 marks a padding token, whose outputs are
 *               left as they are
 *   out         [n_tokens, n_heads, head_dim] dtype, tokens plan->out_stride apart;
 *               it must not overlap q
 *   lse         [n_tokens, n_heads] fp32, contiguous, or NULL
 *   sm_scale    any number that times log2(e) is finite; negative and 0 too
 * Device-data errors set status bits instead of faulting: a position below -1,
 * a row outside the table or a position past its pages: DDTREE_ST_BAD_LENGTH,
 * out 0 and lse -inf; a page outside [0, n_pages): DDTREE_ST_BAD_INDEX, its
 * keys are dropped (out 0 and lse -inf when none is left); a bounded wait
 * inside the kernel that expired: DDTREE_ST_TIMEOUT, and the outputs are not
 * valid.
 * Errors: DDTREE_EINVAL (also a plan that was made for another cache shape),
 * DDTREE_EWORKSPACE, DDTREE_EUNSUPPORTED, DDTREE_ELAUNCH.
 */
DDTREE_API int ddtree_draft_attention(const ddtree_draft_plan_t* plan, const void* q, const ddtree_draft_cache_t* cache,
                                      const int32_t* page_table, int table_rows, int table_stride,
                                      const int32_t* token_rows, const int32_t* positions, float sm_scale, void* out,
                                      float* lse, void* workspace, size_t workspace_bytes,
                                      struct CUstream_st* stream);

#ifdef __cplusplus
}
#endif

#endif /* DDTREE_DRAFT_H_ */
