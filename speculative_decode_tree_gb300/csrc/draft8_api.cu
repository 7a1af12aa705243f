// Host side of the drafter's 8-bit cache (include/ddtree_draft8.h): plan,
// argument checks and launches.
#include <math.h>
#include <string.h>

#include "common.cuh"
#include "../../include/ddtree_draft8.h"

namespace ddtree {
namespace {

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool row_ok(const void* p) { return p && aligned(p, 16); }
inline bool stride_ok(int64_t s, int64_t least) { return s >= least && s % 8 == 0; }
inline bool dtype_ok(int dtype) { return dtype == DDTREE_BF16 || dtype == DDTREE_FP16; }

bool cache_ok(const ddtree_draft8_cache_t* c) {
  if (!c || !row_ok(c->k) || !row_ok(c->v) || !c->k_scale || !aligned(c->k_scale, 4) || !c->v_scale || !aligned(c->v_scale, 4))
    return false;
  if (c->page_size < 1 || c->page_size > DDTREE_MAX_PAGE_SIZE || c->n_pages < 1 || c->n_pages > INT32_MAX / c->page_size)
    return false;
  if (c->n_kv_heads < 1 || c->n_kv_heads > DDTREE_MAX_HEADS) return false;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return false;
  if (c->block_tokens < 1 || c->block_tokens > c->page_size || c->block_tokens > DDTREE_DRAFT8_MAX_BLOCK / c->head_dim)
    return false;
  for (int64_t s : {c->page_stride, c->token_stride, c->head_stride})
    if (s < c->head_dim || s % 16 || s / 16 > UINT32_MAX) return false;
  return true;
}

inline int blocks_of(const ddtree_draft8_cache_t* c) { return (c->page_size + c->block_tokens - 1) / c->block_tokens; }

int device_ok(DevInfo* info) {
  const int rc = current_device_info(info);
  if (rc != DDTREE_OK) return rc;
  return info->major == 10 && info->minor == 3 ? DDTREE_OK : DDTREE_EUNSUPPORTED;
}

bool sizes_ok(int n_tokens, int n_heads, int n_kv_heads, int head_dim, int dtype, int page_size, int block_tokens, int window,
              int n_sinks) {
  return n_tokens >= 1 && n_tokens <= DDTREE_DRAFT_MAX_TOKENS && n_kv_heads >= 1 && n_kv_heads <= DDTREE_MAX_HEADS &&
         n_heads >= n_kv_heads && n_heads % n_kv_heads == 0 && n_heads / n_kv_heads <= DDTREE_DRAFT_MAX_GROUP &&
         (head_dim == 64 || head_dim == 128 || head_dim == 256) && dtype_ok(dtype) && page_size >= 1 &&
         page_size <= DDTREE_MAX_PAGE_SIZE && block_tokens >= 1 && block_tokens <= page_size &&
         block_tokens <= DDTREE_DRAFT8_MAX_BLOCK / head_dim && window >= 0 && n_sinks >= 0;
}

inline int row_tiles_of(int group) { return (group + 15) / 16; }

bool plan_ok(const ddtree_draft8_plan_t* p) {
  if (!p || !sizes_ok(p->n_tokens, p->n_heads, p->n_kv_heads, p->head_dim, p->dtype, p->page_size, p->block_tokens, p->window, p->n_sinks))
    return false;
  if (p->row_tiles != row_tiles_of(p->n_heads / p->n_kv_heads) || p->tile_keys != draft8_tile_keys(p->head_dim) || p->n_shares < 1 ||
      p->n_shares > 65535 || p->workspace_bytes != draft8_workspace_bytes(p->head_dim, p->n_shares))
    return false;
  const int64_t width = (int64_t)p->n_heads * p->head_dim;
  for (int64_t s : {p->q_stride, p->out_stride})
    if (s != 0 && (s < width || s % 8)) return false;
  return true;
}

}  // namespace
}  // namespace ddtree

using namespace ddtree;

extern "C" int ddtree_draft8_append(int64_t n_tokens, int n_heads, int dtype, const ddtree_draft8_cache_t* cache,
                                    const ddtree_rope_t* rope, const void* q, int64_t q_stride, const void* k,
                                    int64_t k_stride, const void* v, int64_t v_stride, const void* q_weight,
                                    const void* k_weight, float eps, const int32_t* positions, const int32_t* slots,
                                    void* q_out, int64_t q_out_stride, uint32_t* status, struct CUstream_st* stream) {
  if (n_tokens < 0 || n_tokens > DDTREE_APPEND_MAX_TOKENS || n_heads < 0 || n_heads > DDTREE_DRAFT_MAX_HEADS)
    return DDTREE_EINVAL;
  if (!dtype_ok(dtype) || !cache_ok(cache) || !rope || rope->rot_dim < 16 || rope->rot_dim > cache->head_dim ||
      rope->rot_dim % 16 || rope->interleaved < 0 || rope->interleaved > 1 || !isfinite(rope->mscale) || !(eps >= 0.f) ||
      !isfinite(eps))
    return DDTREE_EINVAL;
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(status, 4)) return DDTREE_EINVAL;
  if (n_tokens == 0) {  // nothing to read: the tokens' pointers are not looked at
    DevInfo info;
    return device_ok(&info);
  }
  const int64_t kv_width = (int64_t)cache->n_kv_heads * cache->head_dim, q_width = (int64_t)n_heads * cache->head_dim;
  if (!row_ok(k) || !row_ok(v) || !stride_ok(k_stride, kv_width) || !stride_ok(v_stride, kv_width)) return DDTREE_EINVAL;
  if (!positions || !aligned(positions, 4) || !slots || !aligned(slots, 4)) return DDTREE_EINVAL;
  if (n_heads > 0) {
    if (!row_ok(q) || !row_ok(q_out) || !stride_ok(q_stride, q_width) || !stride_ok(q_out_stride, q_width)) return DDTREE_EINVAL;
    if (q == q_out && q_stride != q_out_stride) return DDTREE_EINVAL;
  }
  DevInfo info;
  const int rc = device_ok(&info);
  if (rc != DDTREE_OK) return rc;

  Draft8AppendArgs a;
  memset(&a, 0, sizeof(a));
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_weight = static_cast<const uint16_t*>(q_weight);
  a.k_weight = static_cast<const uint16_t*>(k_weight);
  a.positions = positions;
  a.slots = slots;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_cache = static_cast<uint8_t*>(cache->k);
  a.v_cache = static_cast<uint8_t*>(cache->v);
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.status = status;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out_stride = q_out_stride;
  a.page_stride = cache->page_stride;
  a.token_stride = cache->token_stride;
  a.head_stride = cache->head_stride;
  a.total_slots = cache->n_pages * cache->page_size;
  a.eps = eps;
  a.n_tokens = (int32_t)n_tokens;
  a.n_heads = n_heads;
  a.n_kv_heads = cache->n_kv_heads;
  a.head_dim = cache->head_dim;
  a.page_size = cache->page_size;
  a.block_tokens = cache->block_tokens;
  a.blocks = blocks_of(cache);
  a.page = make_divider(cache->page_size);
  a.block = make_divider(cache->block_tokens);
  a.dtype = dtype;
  a.rope.rot_dim = rope->rot_dim;
  a.rope.interleaved = rope->interleaved;
  a.rope.mscale = rope->mscale;
  memcpy(a.rope.turns, rope->turns, sizeof(a.rope.turns));
  if (launch_draft8_append(a, info.sms, (cudaStream_t)stream) != cudaSuccess) {
    cudaGetLastError();
    return DDTREE_ELAUNCH;
  }
  return DDTREE_OK;
}

extern "C" int ddtree_draft8_read(int64_t n_rows, int dtype, const ddtree_draft8_cache_t* cache, const int32_t* slots,
                                  void* k_out, int64_t k_out_stride, void* v_out, int64_t v_out_stride,
                                  uint32_t* status, struct CUstream_st* stream) {
  if (n_rows < 0 || n_rows > DDTREE_APPEND_MAX_TOKENS || !dtype_ok(dtype) || !cache_ok(cache) || !aligned(status, 4))
    return DDTREE_EINVAL;
  if (n_rows == 0) {
    DevInfo info;
    return device_ok(&info);
  }
  const int64_t width = (int64_t)cache->n_kv_heads * cache->head_dim;
  if (!slots || !aligned(slots, 4) || (!k_out && !v_out) || !aligned(k_out, 16) || !aligned(v_out, 16) || k_out == v_out)
    return DDTREE_EINVAL;
  if ((k_out && !stride_ok(k_out_stride, width)) || (v_out && !stride_ok(v_out_stride, width))) return DDTREE_EINVAL;
  DevInfo info;
  const int rc = device_ok(&info);
  if (rc != DDTREE_OK) return rc;

  Draft8ReadArgs a;
  memset(&a, 0, sizeof(a));
  a.k_cache = static_cast<const uint8_t*>(cache->k);
  a.v_cache = static_cast<const uint8_t*>(cache->v);
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.slots = slots;
  a.k_out = static_cast<uint16_t*>(k_out);
  a.v_out = static_cast<uint16_t*>(v_out);
  a.status = status;
  a.k_out_stride = k_out_stride;
  a.v_out_stride = v_out_stride;
  a.page_stride = cache->page_stride;
  a.token_stride = cache->token_stride;
  a.head_stride = cache->head_stride;
  a.total_slots = cache->n_pages * cache->page_size;
  a.page = make_divider(cache->page_size);
  a.block = make_divider(cache->block_tokens);
  a.n_rows = (int32_t)n_rows;
  a.row_pieces = (int32_t)(width / 8);
  a.n_kv_heads = cache->n_kv_heads;
  a.head_dim = cache->head_dim;
  a.page_size = cache->page_size;
  a.blocks = blocks_of(cache);
  a.dtype = dtype;
  if (launch_draft8_read(a, info.sms, (cudaStream_t)stream) != cudaSuccess) {
    cudaGetLastError();
    return DDTREE_ELAUNCH;
  }
  return DDTREE_OK;
}

extern "C" int ddtree_draft8_attention_plan(int n_tokens, int n_heads, const ddtree_draft8_cache_t* cache, int dtype,
                                            int window, int n_sinks, int num_sms, ddtree_draft8_plan_t* plan) {
  if (!plan || !cache_ok(cache) || num_sms < 0 || num_sms > 4096) return DDTREE_EINVAL;
  if (!sizes_ok(n_tokens, n_heads, cache->n_kv_heads, cache->head_dim, dtype, cache->page_size, cache->block_tokens, window, n_sinks))
    return DDTREE_EINVAL;
  if (num_sms == 0) {
    DevInfo info;
    const int rc = current_device_info(&info);
    if (rc != DDTREE_OK) return rc;
    num_sms = info.sms;
  }
  ddtree_draft8_plan_t p;
  memset(&p, 0, sizeof(p));
  p.n_tokens = n_tokens;
  p.n_heads = n_heads;
  p.n_kv_heads = cache->n_kv_heads;
  p.head_dim = cache->head_dim;
  p.dtype = dtype;
  p.page_size = cache->page_size;
  p.block_tokens = cache->block_tokens;
  p.window = window;
  p.n_sinks = n_sinks;
  p.row_tiles = row_tiles_of(n_heads / cache->n_kv_heads);
  p.tile_keys = draft8_tile_keys(p.head_dim);
  p.n_shares = draft8_shares(p.head_dim, num_sms);
  p.workspace_bytes = draft8_workspace_bytes(p.head_dim, p.n_shares);
  *plan = p;
  return DDTREE_OK;
}

extern "C" size_t ddtree_draft8_attention_workspace_size(const ddtree_draft8_plan_t* plan) {
  return plan ? (size_t)plan->workspace_bytes : 0;
}

extern "C" int ddtree_draft8_attention(const ddtree_draft8_plan_t* plan, const void* q,
                                       const ddtree_draft8_cache_t* cache, const int32_t* page_table, int table_rows,
                                       int table_stride, const int32_t* token_rows, const int32_t* positions,
                                       float sm_scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                       struct CUstream_st* stream) {
  if (!plan_ok(plan) || !cache_ok(cache)) return DDTREE_EINVAL;
  if (plan->n_kv_heads != cache->n_kv_heads || plan->head_dim != cache->head_dim || plan->page_size != cache->page_size ||
      plan->block_tokens != cache->block_tokens)
    return DDTREE_EINVAL;
  if (!q || !aligned(q, 16) || !page_table || !aligned(page_table, 4) || !aligned(token_rows, 4) || !positions ||
      !aligned(positions, 4) || !out || !aligned(out, 16) || !aligned(lse, 4) || !workspace || !aligned(workspace, 256))
    return DDTREE_EINVAL;
  if (table_rows < 1 || table_stride < 1 || (!token_rows && table_rows < plan->n_tokens) || q == out) return DDTREE_EINVAL;
  const float scale_log2 = sm_scale * 1.4426950408889634f;
  if (!isfinite(scale_log2)) return DDTREE_EINVAL;
  if ((int64_t)workspace_bytes < plan->workspace_bytes) return DDTREE_EWORKSPACE;
  DevInfo info;
  const int rc = device_ok(&info);
  if (rc != DDTREE_OK) return rc;

  const int64_t width = (int64_t)plan->n_heads * plan->head_dim;
  Draft8AttnArgs a;
  memset(&a, 0, sizeof(a));
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint8_t*>(cache->k);
  a.v = static_cast<const uint8_t*>(cache->v);
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.table = page_table;
  a.token_rows = token_rows;
  a.positions = positions;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.ws = static_cast<uint8_t*>(workspace);
  a.q_stride = plan->q_stride ? plan->q_stride : width;
  a.out_stride = plan->out_stride ? plan->out_stride : width;
  a.page_step = (uint32_t)(cache->page_stride / 16);
  a.token_step = (uint32_t)(cache->token_stride / 16);
  a.head_step = (uint32_t)(cache->head_stride / 16);
  a.n_pages = (int32_t)cache->n_pages;
  a.scale_log2 = scale_log2;
  a.page = make_divider(cache->page_size);
  a.block = make_divider(cache->block_tokens);
  a.n_tokens = plan->n_tokens;
  a.n_heads = plan->n_heads;
  a.n_kv_heads = plan->n_kv_heads;
  a.group = plan->n_heads / plan->n_kv_heads;
  a.head_dim = plan->head_dim;
  a.dtype = plan->dtype;
  a.page_size = plan->page_size;
  a.blocks = blocks_of(cache);
  a.row_tiles = plan->row_tiles;
  a.unit_heads = plan->n_kv_heads * plan->row_tiles;
  a.window = plan->window;
  a.n_sinks = plan->n_sinks;
  a.table_rows = table_rows;
  a.table_stride = table_stride;
  a.n_shares = plan->n_shares;
  while (a.bundle_log2 < 3 && a.unit_heads % (2 << a.bundle_log2) == 0 && (2 << a.bundle_log2) <= a.n_shares) ++a.bundle_log2;
  if (launch_draft8_attention(a, (cudaStream_t)stream) != cudaSuccess) {
    cudaGetLastError();
    return DDTREE_ELAUNCH;
  }
  return DDTREE_OK;
}
