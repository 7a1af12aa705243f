// Host side of the step maps (include/ddtree_maps.h): argument checks and the
// launch.
#include <string.h>

#include "common.cuh"
#include "../../include/ddtree_maps.h"

namespace {
inline bool ok4(const void* p) { return p && ((uintptr_t)p & 3) == 0; }
inline bool opt4(const void* p) { return ((uintptr_t)p & 3) == 0; }
}  // namespace

using namespace ddtree;

extern "C" int ddtree_step_maps(int batch, int max_new, int page_size, int64_t n_pages, int32_t* page_table,
                                int table_rows, int table_stride, const int32_t* table_row,
                                const int32_t* prefix_lens, const int32_t* new_lens, const int32_t* tree_parent,
                                const int32_t* pages_held, const int32_t* free_pages, int n_free,
                                const int32_t* free_head, int32_t* pages_held_out, int32_t* free_head_out,
                                int32_t* kv_indptr, int32_t* kv_indices, int64_t capacity, int32_t* new_indptr,
                                int32_t* new_slots, int32_t* positions, int32_t* token_rows, uint32_t* status,
                                struct CUstream_st* stream) {
  if (batch < 1 || batch > DDTREE_MAX_BATCH || max_new < 1 || max_new > DDTREE_MAX_NODES) return DDTREE_EINVAL;
  if (page_size < 1 || page_size > DDTREE_MAX_PAGE_SIZE || n_pages < 1 || n_pages > INT32_MAX / page_size)
    return DDTREE_EINVAL;
  if (table_rows < 1 || table_stride < 1 || (!table_row && table_rows < batch)) return DDTREE_EINVAL;
  if (!ok4(page_table) || !opt4(table_row) || !ok4(prefix_lens) || !opt4(new_lens) || !opt4(tree_parent) ||
      !ok4(kv_indptr) || !opt4(kv_indices) || !opt4(new_indptr) || !ok4(new_slots) || !ok4(positions) ||
      !opt4(token_rows) || !opt4(status))
    return DDTREE_EINVAL;
  if (kv_indices ? capacity < 0 : capacity != 0) return DDTREE_EINVAL;
  const bool grow = pages_held != nullptr;
  if (grow) {
    if (!ok4(pages_held) || !ok4(free_head) || !ok4(pages_held_out) || !ok4(free_head_out) || n_free < 0 ||
        (n_free > 0 && !ok4(free_pages)))
      return DDTREE_EINVAL;
    // Every CTA reads the inputs while one writes the outputs.
    if (pages_held == pages_held_out || free_head == free_head_out) return DDTREE_EINVAL;
  } else if (free_pages || n_free || free_head || pages_held_out || free_head_out) {
    return DDTREE_EINVAL;
  }
  DevInfo info;
  int rc = current_device_info(&info);
  if (rc != DDTREE_OK) return rc;
  if (info.major != 10 || info.minor != 3) return DDTREE_EUNSUPPORTED;

  MapsArgs a;
  memset(&a, 0, sizeof(a));
  a.table = page_table;
  a.table_row = table_row;
  a.prefix_lens = prefix_lens;
  a.new_lens = new_lens;
  a.parent = tree_parent;
  a.held = pages_held;
  a.free_pages = free_pages;
  a.free_head = free_head;
  a.held_out = pages_held_out;
  a.free_head_out = free_head_out;
  a.kv_indptr = kv_indptr;
  a.kv_indices = kv_indices;
  a.new_indptr = new_indptr;
  a.new_slots = new_slots;
  a.positions = positions;
  a.token_rows = token_rows;
  a.status = status;
  a.n_pages = n_pages;
  a.capacity = capacity;
  a.batch = batch;
  a.max_new = max_new;
  a.page_size = page_size;
  a.page = make_divider(page_size);
  a.table_rows = table_rows;
  a.table_stride = table_stride;
  a.n_free = n_free;
  if (launch_maps(a, info.sms, (cudaStream_t)stream) != cudaSuccess) {
    cudaGetLastError();
    return DDTREE_ELAUNCH;
  }
  return DDTREE_OK;
}
