/*
 * Causal attention over whole prompts, packed one behind the other: what the
 * drafter runs when it takes in a prompt or a chunk of one ("Chunk 66.0",
 * magik.net seg_66/chunk_0: the drafter has sliding-window attention and KV
 * caching; its cache has to be filled before it can propose).
 *
 * Sequence b has the query rows q_indptr[b] .. q_indptr[b+1] - 1 and the key
 * rows k_indptr[b] .. k_indptr[b+1] - 1.  Its queries are the last of its
 * keys: with nq and nk of them, query i stands at position p = nk - nq + i and
 * sees
 *     K(i) = { j < nk :  j <= p  and  (j > p - window  or  j < n_sinks) }   (window 0: all j <= p)
 *     out[i, h] = sum_j softmax_j(sm_scale <q[i, h], k_j>) v_j,
 *     lse[i, h] = ln sum_j exp(sm_scale <q[i, h], k_j>)
 * with the key head h / (n_heads / n_kv_heads): the rows that the drafter's
 * one-token attention (ddtree_draft.h) would give, one after the other.  A
 * query that sees nothing (more queries than keys) has out 0 and lse -inf.
 * A key that a query does not see has no part in its row, whatever it holds
 * (NaN and infinities too).  Where some queries of a work item see a value that
 * is no number and others do not, the item's rows are computed again key by key,
 * with probabilities that are not rounded: the others' rows are within the same
 * bounds then, but not to the bit what they are without that value, and the call
 * takes longer (16,384 tokens of 16 + 2 heads of 128 columns 0.65 ms; with a NaN
 * in the last value 6 ms, in the first one, which most rows see, 150 ms; what
 * keys and queries hold costs nothing).  A row that sees nothing but scores of
 * -inf is no number, nor is one that sees an infinite value with a probability
 * below 2^-126.
 *
 * Scores, maxima and sums are in 32 bits; a probability is rounded to the
 * inputs' type (half a step of it) where it meets V, while the sums take it
 * unrounded, and fp16 probabilities carry a factor of 2^10, so that keys down
 * to 2^-34 of the largest count.  An output is rounded once.  Equal inputs give
 * equal bits.  The tensor cores cut their sums off at 32 bits, which takes 6e-9 of
 * sum p |v| for each key: rows of many keys are summed in parts of 16,384 (where
 * rows of the plan may see more than 32,768), so that this stays below 2e-4.
 *
 * Conventions as in ddtree_verify.h.
 */
#ifndef DDTREE_PROMPT_H_
#define DDTREE_PROMPT_H_

#include "ddtree_draft.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DDTREE_PROMPT_MAX_ROWS (1 << 24)

/* Fields are outputs of ddtree_prompt_attention_plan except wait_limit_us and
 * the strides, which the caller may set afterwards (0: 2 s, contiguous). */
typedef struct ddtree_prompt_plan {
  int32_t batch, n_heads, n_kv_heads, head_dim, dtype;
  int32_t window, n_sinks;
  int32_t q_rows, k_rows;      /* rows of the packed buffers                       */
  int32_t wait_limit_us;       /* bound of each wait inside the kernel for a copy, a
                                  product or another warp; one that expires sets
                                  DDTREE_ST_TIMEOUT, and the call ends without it (a
                                  CTA within a few such bounds, and 2 s for what is
                                  on its way); below 1 ms waits poll  */
  int32_t tile_tokens;         /* query tokens of a work item                      */
  int32_t max_items;           /* work items of the fullest batch                  */
  int64_t q_stride, k_stride, v_stride, out_stride;  /* elements between rows, multiples of 8 */
  int64_t workspace_bytes;
} ddtree_prompt_plan_t;

/*
 * batch 1 .. DDTREE_MAX_BATCH; q_rows, k_rows 1 .. DDTREE_PROMPT_MAX_ROWS, the
 * rows of the buffers (the sequences may fill less of them); n_kv_heads 1 ..
 * DDTREE_MAX_HEADS, n_heads a multiple of it, at most DDTREE_DRAFT_MAX_GROUP
 * times; head_dim 64, 128 or 256; dtype DDTREE_BF16 or DDTREE_FP16; window and
 * n_sinks 0 .. 2^31-1.  Lengths are on the device, so the kernel's form for short
 * sequences goes by q_rows and batch: buffers much larger than what is in them
 * cost short prompts time (200 of 20 to 30 tokens 31 us, in buffers of 65,536 rows
 * 43).  Host only.  Errors: DDTREE_EINVAL.
 */
DDTREE_API int ddtree_prompt_attention_plan(int batch, int q_rows, int k_rows, int n_heads, int n_kv_heads, int head_dim,
                                            int dtype, int window, int n_sinks, ddtree_prompt_plan_t* plan);

/* Workspace bytes for a plan (a multiple of 256; 256-byte aligned buffer): the
 * 256-byte status block (read with ddtree_verify_mla_check), a word for each
 * work item, and where rows may see more than 32,768 keys 64 or 128 KB for each
 * of up to 320 thread blocks (20 MB at most).  It keeps nothing between calls; calls that may overlap on
 * the GPU need a workspace each.  0 for a null plan. */
DDTREE_API size_t ddtree_prompt_attention_workspace_size(const ddtree_prompt_plan_t* plan);

/*
 *   q         [q_rows, n_heads, head_dim] dtype, rows plan->q_stride apart
 *   k, v      [k_rows, n_kv_heads, head_dim] dtype, rows plan->k_stride, v_stride
 *             apart (the three may be parts of one projection)
 *   q_indptr  [batch + 1] int32, 0 <= q_indptr[0] <= ... <= q_rows
 *   k_indptr  [batch + 1] int32, likewise; NULL: q_indptr (prompts without an
 *             earlier context)
 *   out       [q_rows, n_heads, head_dim] dtype, rows plan->out_stride apart; rows
 *             of no sequence are left as they are.  It must not overlap q, k, v.
 *   lse       [q_rows, n_heads] fp32, contiguous, or NULL
 *   sm_scale  any number that times log2(e) is finite
 * Device-data errors set status bits instead of faulting: a sequence whose
 * indptr entries decrease or leave the buffers: DDTREE_ST_BAD_LENGTH, and no
 * sequence's rows are written; a bounded wait that expired:
 * DDTREE_ST_TIMEOUT, and the outputs are not valid.
 * Errors: DDTREE_EINVAL, DDTREE_EWORKSPACE, DDTREE_EUNSUPPORTED, DDTREE_ELAUNCH.
 */
DDTREE_API int ddtree_prompt_attention(const ddtree_prompt_plan_t* plan, const void* q, const void* k, const void* v,
                                       const int32_t* q_indptr, const int32_t* k_indptr, float sm_scale, void* out,
                                       float* lse, void* workspace, size_t workspace_bytes, struct CUstream_st* stream);

#ifdef __cplusplus
}
#endif

#endif /* DDTREE_PROMPT_H_ */
