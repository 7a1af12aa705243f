// Host side of the prompt attention (include/ddtree_prompt.h): plan, argument
// checks and the launch.
#include <math.h>
#include <string.h>

#include "common.cuh"
#include "../../include/ddtree_prompt.h"

namespace ddtree {
namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 32;  // elements between rows: what a tensor map takes

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool sizes_ok(int batch, int q_rows, int k_rows, int n_heads, int n_kv_heads, int head_dim, int dtype, int window, int n_sinks) {
  return batch >= 1 && batch <= DDTREE_MAX_BATCH && q_rows >= 1 && q_rows <= DDTREE_PROMPT_MAX_ROWS && k_rows >= 1 &&
         k_rows <= DDTREE_PROMPT_MAX_ROWS && n_kv_heads >= 1 && n_kv_heads <= DDTREE_MAX_HEADS && n_heads >= n_kv_heads &&
         n_heads % n_kv_heads == 0 && n_heads / n_kv_heads <= DDTREE_DRAFT_MAX_GROUP &&
         (head_dim == 64 || head_dim == 128 || head_dim == 256) && (dtype == DDTREE_BF16 || dtype == DDTREE_FP16) && window >= 0 &&
         n_sinks >= 0;
}

// Work items of the fullest batch: a tile for every tile_tokens rows, and one
// more that each sequence may leave unfilled.
int64_t items_of(int batch, int q_rows, int n_kv_heads, int tile_tokens) {
  return ((int64_t)q_rows / tile_tokens + batch) * n_kv_heads;
}

int64_t words_end(int64_t items) { return 256 + (items * 4 + 255) / 256 * 256; }

int64_t workspace_of(const ddtree_prompt_plan_t& p, int64_t items) {
  return words_end(items) + prompt_fold_bytes(p.k_rows, p.head_dim, p.n_heads / p.n_kv_heads, p.window, p.n_sinks, p.tile_tokens, items);
}

bool plan_ok(const ddtree_prompt_plan_t* p) {
  if (!p || !sizes_ok(p->batch, p->q_rows, p->k_rows, p->n_heads, p->n_kv_heads, p->head_dim, p->dtype, p->window, p->n_sinks))
    return false;
  if (p->tile_tokens != prompt_tile_tokens(p->batch, p->q_rows, p->n_heads / p->n_kv_heads, p->head_dim) || p->wait_limit_us < 0) return false;
  const int64_t items = items_of(p->batch, p->q_rows, p->n_kv_heads, p->tile_tokens);
  if (items > INT32_MAX || p->max_items != items || p->workspace_bytes != workspace_of(*p, items)) return false;
  const int64_t width = (int64_t)p->n_heads * p->head_dim, kv_width = (int64_t)p->n_kv_heads * p->head_dim;
  for (int64_t s : {p->q_stride, p->out_stride})
    if (s != 0 && (s < width || s % 8 || s > kMaxStride)) return false;
  for (int64_t s : {p->k_stride, p->v_stride})
    if (s != 0 && (s < kv_width || s % 8 || s > kMaxStride)) return false;
  return true;
}

}  // namespace
}  // namespace ddtree

using namespace ddtree;

extern "C" int ddtree_prompt_attention_plan(int batch, int q_rows, int k_rows, int n_heads, int n_kv_heads, int head_dim,
                                            int dtype, int window, int n_sinks, ddtree_prompt_plan_t* plan) {
  if (!plan || !sizes_ok(batch, q_rows, k_rows, n_heads, n_kv_heads, head_dim, dtype, window, n_sinks)) return DDTREE_EINVAL;
  ddtree_prompt_plan_t p;
  memset(&p, 0, sizeof(p));
  p.batch = batch;
  p.n_heads = n_heads;
  p.n_kv_heads = n_kv_heads;
  p.head_dim = head_dim;
  p.dtype = dtype;
  p.window = window;
  p.n_sinks = n_sinks;
  p.q_rows = q_rows;
  p.k_rows = k_rows;
  p.tile_tokens = prompt_tile_tokens(batch, q_rows, n_heads / n_kv_heads, head_dim);
  const int64_t items = items_of(batch, q_rows, n_kv_heads, p.tile_tokens);
  if (items > INT32_MAX) return DDTREE_EINVAL;
  p.max_items = (int32_t)items;
  p.workspace_bytes = workspace_of(p, items);
  *plan = p;
  return DDTREE_OK;
}

extern "C" size_t ddtree_prompt_attention_workspace_size(const ddtree_prompt_plan_t* plan) {
  return plan ? (size_t)plan->workspace_bytes : 0;
}

extern "C" int ddtree_prompt_attention(const ddtree_prompt_plan_t* plan, const void* q, const void* k, const void* v,
                                       const int32_t* q_indptr, const int32_t* k_indptr, float sm_scale, void* out,
                                       float* lse, void* workspace, size_t workspace_bytes, struct CUstream_st* stream) {
  if (!plan_ok(plan)) return DDTREE_EINVAL;
  for (const void* p : {q, k, v, (const void*)out})
    if (!p || !aligned(p, 16)) return DDTREE_EINVAL;
  if (!q_indptr || !aligned(q_indptr, 4) || !aligned(k_indptr, 4) || !aligned(lse, 4) || !workspace || !aligned(workspace, 256) ||
      out == q || out == k || out == v)
    return DDTREE_EINVAL;
  const float scale_log2 = sm_scale * 1.4426950408889634f;
  if (!isfinite(scale_log2)) return DDTREE_EINVAL;
  if ((int64_t)workspace_bytes < plan->workspace_bytes) return DDTREE_EWORKSPACE;
  DevInfo info;
  const int rc = current_device_info(&info);
  if (rc != DDTREE_OK) return rc;
  if (info.major != 10 || info.minor != 3) return DDTREE_EUNSUPPORTED;

  const int64_t width = (int64_t)plan->n_heads * plan->head_dim, kv_width = (int64_t)plan->n_kv_heads * plan->head_dim;
  PromptArgs a;
  memset(&a, 0, sizeof(a));
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_indptr = q_indptr;
  a.k_indptr = k_indptr ? k_indptr : q_indptr;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.status = static_cast<uint32_t*>(workspace);
  a.words = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + 256);
  const int64_t folds_at = words_end(plan->max_items);
  if (plan->workspace_bytes > folds_at) a.folds = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + folds_at);
  a.q_stride = plan->q_stride ? plan->q_stride : width;
  a.k_stride = plan->k_stride ? plan->k_stride : kv_width;
  a.v_stride = plan->v_stride ? plan->v_stride : kv_width;
  a.out_stride = plan->out_stride ? plan->out_stride : width;
  a.scale_log2 = scale_log2;
  a.wait_ns = plan->wait_limit_us > 0 ? (uint64_t)plan->wait_limit_us * 1000ull : 2000000000ull;
  a.batch = plan->batch;
  a.n_heads = plan->n_heads;
  a.n_kv_heads = plan->n_kv_heads;
  a.group = plan->n_heads / plan->n_kv_heads;
  a.head_dim = plan->head_dim;
  a.dtype = plan->dtype;
  // A window of all rows is none; positions may be below 0, and less a larger one they would pass 32 bits.
  a.window = plan->window >= DDTREE_PROMPT_MAX_ROWS ? 0 : plan->window;
  a.n_sinks = plan->n_sinks;
  a.q_rows = plan->q_rows;
  a.k_rows = plan->k_rows;
  a.tile_tokens = plan->tile_tokens;
  a.max_items = plan->max_items;
  if (launch_prompt(a, info.sms, (cudaStream_t)stream) != cudaSuccess) {
    cudaGetLastError();
    return DDTREE_ELAUNCH;
  }
  return DDTREE_OK;
}
