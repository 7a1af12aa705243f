// Host side of the drafter's attention (include/ddtree_draft.h): plan,
// argument checks and the launch.
#include <math.h>
#include <string.h>

#include "common.cuh"
#include "../../include/ddtree_draft.h"

namespace ddtree {
namespace {

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool sizes_ok(int n_tokens, int n_heads, int n_kv_heads, int head_dim, int dtype, int page_size, int window, int n_sinks) {
  return n_tokens >= 1 && n_tokens <= DDTREE_DRAFT_MAX_TOKENS && n_kv_heads >= 1 && n_kv_heads <= DDTREE_MAX_HEADS &&
         n_heads >= n_kv_heads && n_heads % n_kv_heads == 0 && n_heads / n_kv_heads <= DDTREE_DRAFT_MAX_GROUP &&
         (head_dim == 64 || head_dim == 128 || head_dim == 256) && (dtype == DDTREE_BF16 || dtype == DDTREE_FP16) &&
         page_size >= 1 && page_size <= DDTREE_MAX_PAGE_SIZE && window >= 0 && n_sinks >= 0;
}

bool plan_ok(const ddtree_draft_plan_t* p) {
  if (!p || !sizes_ok(p->n_tokens, p->n_heads, p->n_kv_heads, p->head_dim, p->dtype, p->page_size, p->window, p->n_sinks))
    return false;
  if (p->row_tile != draft_row_tile(p->n_heads / p->n_kv_heads, p->head_dim) || p->tile_keys != draft_tile_keys(p->row_tile, p->head_dim) ||
      p->n_shares < 1 || p->n_shares > 65535 || p->wait_limit_us < 0)
    return false;
  if (p->workspace_bytes != draft_workspace_bytes(p->row_tile, p->head_dim, p->n_shares)) return false;
  const int64_t width = (int64_t)p->n_heads * p->head_dim;
  for (int64_t s : {p->q_stride, p->out_stride})
    if (s != 0 && (s < width || s % 8)) return false;
  return true;
}

}  // namespace
}  // namespace ddtree

using namespace ddtree;

extern "C" int ddtree_draft_attention_plan(int n_tokens, int n_heads, const ddtree_draft_cache_t* cache, int window,
                                           int n_sinks, int num_sms, ddtree_draft_plan_t* plan) {
  if (!plan || !draft_cache_ok(cache) || num_sms < 0 || num_sms > 4096) return DDTREE_EINVAL;
  if (!sizes_ok(n_tokens, n_heads, cache->n_kv_heads, cache->head_dim, cache->dtype, cache->page_size, window, n_sinks))
    return DDTREE_EINVAL;
  if (num_sms == 0) {
    DevInfo info;
    const int rc = current_device_info(&info);
    if (rc != DDTREE_OK) return rc;
    num_sms = info.sms;
  }
  ddtree_draft_plan_t p;
  memset(&p, 0, sizeof(p));
  p.n_tokens = n_tokens;
  p.n_heads = n_heads;
  p.n_kv_heads = cache->n_kv_heads;
  p.head_dim = cache->head_dim;
  p.dtype = cache->dtype;
  p.page_size = cache->page_size;
  p.window = window;
  p.n_sinks = n_sinks;
  p.row_tile = draft_row_tile(n_heads / cache->n_kv_heads, p.head_dim);
  p.tile_keys = draft_tile_keys(p.row_tile, p.head_dim);
  p.n_shares = draft_shares(p.row_tile, p.head_dim, num_sms);
  p.workspace_bytes = draft_workspace_bytes(p.row_tile, p.head_dim, p.n_shares);
  *plan = p;
  return DDTREE_OK;
}

extern "C" size_t ddtree_draft_attention_workspace_size(const ddtree_draft_plan_t* plan) {
  return plan ? (size_t)plan->workspace_bytes : 0;
}

extern "C" int ddtree_draft_attention(const ddtree_draft_plan_t* plan, const void* q, const ddtree_draft_cache_t* cache,
                                      const int32_t* page_table, int table_rows, int table_stride,
                                      const int32_t* token_rows, const int32_t* positions, float sm_scale, void* out,
                                      float* lse, void* workspace, size_t workspace_bytes,
                                      struct CUstream_st* stream) {
  if (!plan_ok(plan) || !draft_cache_ok(cache)) return DDTREE_EINVAL;
  if (plan->n_kv_heads != cache->n_kv_heads || plan->head_dim != cache->head_dim || plan->dtype != cache->dtype ||
      plan->page_size != cache->page_size)
    return DDTREE_EINVAL;
  if (!q || !aligned(q, 16) || !page_table || !aligned(page_table, 4) || !aligned(token_rows, 4) || !positions ||
      !aligned(positions, 4) || !out || !aligned(out, 16) || !aligned(lse, 4) || !workspace || !aligned(workspace, 256))
    return DDTREE_EINVAL;
  if (table_rows < 1 || table_stride < 1 || (!token_rows && table_rows < plan->n_tokens) || q == out)
    return DDTREE_EINVAL;
  const float scale_log2 = sm_scale * 1.4426950408889634f;
  if (!isfinite(scale_log2)) return DDTREE_EINVAL;
  if ((int64_t)workspace_bytes < plan->workspace_bytes) return DDTREE_EWORKSPACE;
  DevInfo info;
  const int rc = current_device_info(&info);
  if (rc != DDTREE_OK) return rc;
  if (info.major != 10 || info.minor != 3) return DDTREE_EUNSUPPORTED;

  const int64_t width = (int64_t)plan->n_heads * plan->head_dim;
  DraftAttnArgs a;
  memset(&a, 0, sizeof(a));
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(cache->k);
  a.v = static_cast<const uint16_t*>(cache->v);
  a.table = page_table;
  a.token_rows = token_rows;
  a.positions = positions;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.ws = static_cast<uint8_t*>(workspace);
  a.q_stride = plan->q_stride ? plan->q_stride : width;
  a.out_stride = plan->out_stride ? plan->out_stride : width;
  a.page_stride = cache->page_stride;
  a.token_stride = cache->token_stride;
  a.head_stride = cache->head_stride;
  a.n_pages = cache->n_pages;
  a.scale_log2 = scale_log2;
  a.wait_ns = plan->wait_limit_us > 0 ? (uint64_t)plan->wait_limit_us * 1000ull : 2000000000ull;
  a.n_tokens = plan->n_tokens;
  a.n_heads = plan->n_heads;
  a.n_kv_heads = plan->n_kv_heads;
  a.group = plan->n_heads / plan->n_kv_heads;
  a.head_dim = plan->head_dim;
  a.dtype = plan->dtype;
  a.page_size = plan->page_size;
  a.page = make_divider(plan->page_size);
  a.window = plan->window;
  a.n_sinks = plan->n_sinks;
  a.table_rows = table_rows;
  a.table_stride = table_stride;
  a.row_tile = plan->row_tile;
  a.n_shares = plan->n_shares;
  while (a.bundle_log2 < 3 && plan->n_kv_heads % (2 << a.bundle_log2) == 0 && (2 << a.bundle_log2) <= a.n_shares) ++a.bundle_log2;
  if (launch_draft_attention(a, (cudaStream_t)stream) != cudaSuccess) {
    cudaGetLastError();
    return DDTREE_ELAUNCH;
  }
  return DDTREE_OK;
}
