/*
 * Writing new tokens into the caches: norms, position rotation and the row
 * write in one pass.
 *
 * Verify attention takes rotated queries and finds the tree nodes' rows in the
 * pool ("Chunk 66.0", magik.net seg_66/chunk_0: MLA on a token-granular pool;
 * a row is 512 latent + 64 rope columns).  ddtree_mla_append makes both from
 * what the projections give; ddtree_draft_append does the same for the
 * drafter, which keeps a key and a value cache of its own ("Chunk 66.0": the
 * drafter has sliding-window attention and KV caching).
 *
 * The rotation R(p) turns pair i of a vector's first rot_dim columns by the
 * angle p * f_i.  The angle is kept as a 64-bit fraction of one turn, so the
 * product with any int32 position is exact modulo a turn; sine and cosine are
 * taken in 32 bits of the remainder.  Norms, rotations and products are in 32
 * bits, and every output is rounded once.
 *
 * Conventions as in ddtree_verify.h.
 */
#ifndef DDTREE_APPEND_H_
#define DDTREE_APPEND_H_

#include "ddtree_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DDTREE_ROPE_MAX_PAIRS 128
#define DDTREE_APPEND_MAX_TOKENS (1 << 24)
#define DDTREE_DRAFT_MAX_HEADS 512

#define DDTREE_ROPE_PLAIN  0  /* f_i = theta^(-2i/rot_dim)                                   */
#define DDTREE_ROPE_LINEAR 1  /* positions stretched: f_i / factor                            */
#define DDTREE_ROPE_YARN   2  /* by parts (the YaRN method): pairs that turn more than        */
                              /* beta_fast times over original_positions keep f_i, those      */
                              /* that turn less than beta_slow times get f_i / factor, a      */
                              /* linear ramp over the pair index in between                   */

#define DDTREE_BF16 0
#define DDTREE_FP16 1

/* A rotation, made once on the host by ddtree_rope_init and passed by value
 * into the launches. */
typedef struct ddtree_rope {
  int32_t rot_dim;       /* columns that are rotated (even)                       */
  int32_t interleaved;   /* 1: pairs (2i, 2i+1); 0: pairs (i, i + rot_dim/2)      */
  float mscale;          /* factor on sine and cosine (attention scaling)         */
  int32_t reserved;
  uint64_t turns[DDTREE_ROPE_MAX_PAIRS]; /* f_i / (2 pi) * 2^64, rounded down     */
} ddtree_rope_t;

/*
 * rot_dim 2 .. 256, even; theta > 1; factor >= 1 (ignored by PLAIN); the next
 * three are read by YARN only: beta_fast > beta_slow > 0, original_positions >
 * 2 pi beta_slow (with fewer no pair turns beta_slow times over them).
 * mscale > 0, or 0 for the method's own: 0.1 ln(factor) + 1 for YARN, else 1.
 * Host only.  Errors: DDTREE_EINVAL.
 */
DDTREE_API int ddtree_rope_init(int rot_dim, int interleaved, double theta, int scaling, double factor,
                                int original_positions, double beta_fast, double beta_slow, double mscale,
                                ddtree_rope_t* rope);

/*
 * Latent rows of n_tokens new tokens into the MLA pool, and their queries'
 * rope part:
 *   pool[slots[n]]  = [ norm(kv_new[n, :512]) | R(positions[n]) kv_new[n, 512:] ]
 *   q_out[n, h]     = R(positions[n]) q_rope[n, h]
 * with norm(x) = x / sqrt(mean(x^2) + eps) * latent_weight (x itself when
 * latent_weight is NULL).
 *   n_tokens      0 .. DDTREE_APPEND_MAX_TOKENS (0: nothing happens, and the
 *                 tokens' pointers may be NULL);  n_heads 0 .. DDTREE_MAX_HEADS
 *                 (0: rows only, q_rope and q_out may be NULL)
 *   rope          rot_dim must be 64
 *   kv_new        bf16, 576 columns, rows kv_stride elements apart
 *   latent_weight [512] bf16 or NULL
 *   q_rope        bf16, 64 columns, tokens q_token_stride and heads q_head_stride
 *                 elements apart (e.g. the last 64 columns of a wider projection)
 *   q_out         bf16, likewise with its own strides (e.g. columns 512.. of a
 *                 576-wide query buffer).  It may be q_rope itself with the
 *                 same strides; otherwise the two must not overlap.
 *   positions     [n_tokens] int32; -1 marks a padding token, for which nothing
 *                 is written.  Below -1: DDTREE_ST_BAD_LENGTH, as padding.
 *   slots         [n_tokens] int32 pool rows; -1: the row is not written (the
 *                 queries are).  Others outside [0, pool_rows):
 *                 DDTREE_ST_BAD_INDEX, not written.  Two tokens of a call must
 *                 not name the same row: its contents would be either's, piece
 *                 by piece.
 *   status        uint32, OR-ed (the caller clears it), or NULL
 * Pointers and strides are multiples of 16 bytes (positions, slots, status 4).
 * Errors: DDTREE_EINVAL, DDTREE_EUNSUPPORTED, DDTREE_ELAUNCH.
 */
DDTREE_API int ddtree_mla_append(int64_t n_tokens, int n_heads, const ddtree_rope_t* rope, const ddtree_bf16_t* kv_new,
                                 int64_t kv_stride, const ddtree_bf16_t* latent_weight, float eps,
                                 const ddtree_bf16_t* q_rope, int64_t q_token_stride, int64_t q_head_stride,
                                 const int32_t* positions, const int32_t* slots, ddtree_bf16_t* kv_pool,
                                 int64_t pool_rows, ddtree_bf16_t* q_out, int64_t q_out_token_stride,
                                 int64_t q_out_head_stride, uint32_t* status, struct CUstream_st* stream);

/* The drafter's paged cache: element (page, token, head, column) of k and of v
 * lies page * page_stride + token * token_stride + head * head_stride + column
 * elements behind the pointer, so both orders of tokens and heads are served. */
typedef struct ddtree_draft_cache {
  void* k;               /* 16-byte aligned, dtype elements                       */
  void* v;
  int64_t n_pages;       /* n_pages * page_size <= 2^31 - 1                       */
  int64_t page_stride;   /* elements, multiples of 8                              */
  int64_t token_stride;
  int64_t head_stride;
  int32_t page_size;     /* tokens of a page, 1 .. DDTREE_MAX_PAGE_SIZE, any number */
  int32_t n_kv_heads;    /* 1 .. DDTREE_MAX_HEADS                                 */
  int32_t head_dim;      /* 64, 128 or 256                                        */
  int32_t dtype;         /* DDTREE_BF16 or DDTREE_FP16                            */
} ddtree_draft_cache_t;

/*
 * Queries, keys and values of n_tokens new tokens, for the drafter:
 *   q_out[n, h]           = R(positions[n]) norm(q[n, h], q_weight)
 *   k cache [slots[n], h] = R(positions[n]) norm(k[n, h], k_weight)
 *   v cache [slots[n], h] = v[n, h]
 * norm over the head's head_dim columns as above, left out where the weight is
 * NULL; R turns the first rope->rot_dim columns.
 *   n_tokens      0 .. DDTREE_APPEND_MAX_TOKENS, as above;  n_heads query heads,
 *                 0 .. DDTREE_DRAFT_MAX_HEADS (0: keys and values only, q and
 *                 q_out may be NULL)
 *   rope          rot_dim <= head_dim, a multiple of 16
 *   q, k, v       cache->dtype; tokens *_stride elements apart, heads head_dim
 *                 apart (e.g. parts of one fused projection)
 *   q_out         tokens q_out_stride apart, heads head_dim apart; may be q
 *                 itself with the same stride, otherwise they must not overlap
 *   positions, slots, status as above; slot = page * page_size + token in page
 * Errors: DDTREE_EINVAL, DDTREE_EUNSUPPORTED, DDTREE_ELAUNCH.
 */
DDTREE_API int ddtree_draft_append(int64_t n_tokens, int n_heads, const ddtree_draft_cache_t* cache,
                                   const ddtree_rope_t* rope, const void* q, int64_t q_stride, const void* k,
                                   int64_t k_stride, const void* v, int64_t v_stride, const void* q_weight,
                                   const void* k_weight, float eps, const int32_t* positions, const int32_t* slots,
                                   void* q_out, int64_t q_out_stride, uint32_t* status, struct CUstream_st* stream);

#ifdef __cplusplus
}
#endif

#endif /* DDTREE_APPEND_H_ */
