/*
 * The integer set-up of a decode step: page tables, the verify index layout,
 * slots and positions of the new tokens, all from the requests' lengths.
 *
 * The verify kernels reach a request's keys through kv_indices: its prefix
 * rows, then the rows of its new tokens ("Chunk 66.0", magik.net
 * seg_66/chunk_0: the token-granular, page_size=1 pool).  Serving code keeps a
 * page table per request and a list of free pages; on the pages the host
 * builds what the step needs from them ("Chunk 66.1", magik.net
 * seg_66/chunk_1: CPU tree-build and mask-build).  This call does it on the
 * device, in one launch whose grid does not depend on the lengths, so the whole
 * step can be captured and replayed:
 *
 *   for request b with row r = table_row[b], P = prefix_lens[b] committed
 *   tokens, n = new_lens[b] new ones and h = pages_held[b] pages in the table:
 *     pages     table[r][k] for h <= k < ceil((P+n)/page_size) are taken from
 *               free_pages in order, request by request, from free_head on
 *     rows      row(j) = table[r][j / page_size] * page_size + j % page_size
 *     kv_indptr exclusive sums of P+n;  kv_indices[kv_indptr[b] + j] = row(j)
 *     tokens    packed by request: token new_indptr[b] + i gets
 *                 new_slots  = row(P + i)
 *                 positions  = P + depth(i)   (P + i without a tree)
 *                 token_rows = r
 *               and every entry behind the last token is -1 in all three
 *
 * All or nothing: when a length is out of range (P < 0, n not in [0, max_new],
 * more pages than a table row holds, more pages held than that, kv_indices too
 * small, a row outside the table) the status gets DDTREE_ST_BAD_LENGTH, when
 * the free list runs out DDTREE_ST_NO_PAGES; then the table is left as it was,
 * pages_held_out and free_head_out repeat their inputs, kv_indptr and
 * new_indptr are zero, the token lists are -1 and kv_indices is not written.
 * A page outside [0, n_pages) sets DDTREE_ST_BAD_INDEX and its rows become -1
 * (which the verify kernels drop); a parent that is not -1 or an earlier node
 * sets DDTREE_ST_BAD_PARENT and ends the depth walk there.
 *
 * Conventions as in ddtree_verify.h.
 */
#ifndef DDTREE_MAPS_H_
#define DDTREE_MAPS_H_

#include "ddtree_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 *   batch         requests, 1 .. DDTREE_MAX_BATCH;  max_new 1 .. DDTREE_MAX_NODES
 *   page_size     tokens of a page, 1 .. DDTREE_MAX_PAGE_SIZE (any number);
 *                 n_pages * page_size <= 2^31 - 1
 *   page_table    [table_rows, table_stride] int32, grown in place;
 *                 table_stride is the pages a row can hold
 *   table_row     [batch] int32 row of each request, or NULL (row b).  With a
 *                 free list the rows must differ: two requests that name the
 *                 same row would both write its new pages.
 *   prefix_lens   [batch] int32;  new_lens [batch] int32 or NULL (max_new each)
 *   tree_parent   [batch, max_new] int32 or NULL (a chain)
 *   pages_held    [batch] int32, free_pages [n_free] int32, free_head [1] int32
 *                 (the first page of the list not yet taken), and the outputs
 *                 pages_held_out [batch], free_head_out [1], which must not be
 *                 the same buffers; all five NULL: nothing is taken, every page
 *                 must be in the table
 *   kv_indptr     [batch+1] int32 output
 *   kv_indices    int32 output of `capacity` entries, or NULL
 *   new_indptr    [batch+1] int32 output, or NULL
 *   new_slots, positions  [batch * max_new] int32 outputs;  token_rows likewise, or NULL
 *   status        uint32, OR-ed (the caller clears it), or NULL
 * Errors: DDTREE_EINVAL (null or misaligned pointer, sizes out of range),
 * DDTREE_EUNSUPPORTED, DDTREE_ELAUNCH.
 */
DDTREE_API int ddtree_step_maps(int batch, int max_new, int page_size, int64_t n_pages, int32_t* page_table,
                                int table_rows, int table_stride, const int32_t* table_row,
                                const int32_t* prefix_lens, const int32_t* new_lens, const int32_t* tree_parent,
                                const int32_t* pages_held, const int32_t* free_pages, int n_free,
                                const int32_t* free_head, int32_t* pages_held_out, int32_t* free_head_out,
                                int32_t* kv_indptr, int32_t* kv_indices, int64_t capacity, int32_t* new_indptr,
                                int32_t* new_slots, int32_t* positions, int32_t* token_rows, uint32_t* status,
                                struct CUstream_st* stream);

#ifdef __cplusplus
}
#endif

#endif /* DDTREE_MAPS_H_ */
