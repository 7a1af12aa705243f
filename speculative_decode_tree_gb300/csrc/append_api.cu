// Host side of the append entry points (include/ddtree_append.h): the
// rotation, argument checks and launches.
#include <math.h>
#include <string.h>

#include "common.cuh"

namespace ddtree {
namespace {

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool row_ok(const void* p) { return p && aligned(p, 16); }
inline bool stride_ok(int64_t s, int64_t least) { return s >= least && s % 8 == 0; }

bool rope_ok(const ddtree_rope_t* r) {
  return r && r->rot_dim >= 2 && r->rot_dim <= 2 * DDTREE_ROPE_MAX_PAIRS && r->rot_dim % 2 == 0 &&
         (r->interleaved == 0 || r->interleaved == 1) && isfinite(r->mscale);
}

void copy_rope(const ddtree_rope_t* r, RopeArgs* out) {
  out->rot_dim = r->rot_dim;
  out->interleaved = r->interleaved;
  out->mscale = r->mscale;
  memcpy(out->turns, r->turns, sizeof(out->turns));
}

int device_ok(DevInfo* info) {
  const int rc = current_device_info(info);
  if (rc != DDTREE_OK) return rc;
  return info->major == 10 && info->minor == 3 ? DDTREE_OK : DDTREE_EUNSUPPORTED;
}

}  // namespace

bool draft_cache_ok(const ddtree_draft_cache_t* c) {
  if (!c || !row_ok(c->k) || !row_ok(c->v)) return false;
  if (c->page_size < 1 || c->page_size > DDTREE_MAX_PAGE_SIZE || c->n_pages < 1 || c->n_pages > INT32_MAX / c->page_size)
    return false;
  if (c->n_kv_heads < 1 || c->n_kv_heads > DDTREE_MAX_HEADS) return false;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return false;
  if (c->dtype != DDTREE_BF16 && c->dtype != DDTREE_FP16) return false;
  return stride_ok(c->page_stride, c->head_dim) && stride_ok(c->token_stride, c->head_dim) &&
         stride_ok(c->head_stride, c->head_dim);
}

}  // namespace ddtree

using namespace ddtree;

extern "C" int ddtree_rope_init(int rot_dim, int interleaved, double theta, int scaling, double factor,
                                int original_positions, double beta_fast, double beta_slow, double mscale,
                                ddtree_rope_t* rope) {
  if (!rope || rot_dim < 2 || rot_dim > 2 * DDTREE_ROPE_MAX_PAIRS || rot_dim % 2 || interleaved < 0 || interleaved > 1)
    return DDTREE_EINVAL;
  if (!(theta > 1.0) || !isfinite(theta) || scaling < DDTREE_ROPE_PLAIN || scaling > DDTREE_ROPE_YARN)
    return DDTREE_EINVAL;
  if (scaling != DDTREE_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return DDTREE_EINVAL;
  if (scaling == DDTREE_ROPE_YARN &&
      (original_positions < 1 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !isfinite(beta_fast)))
    return DDTREE_EINVAL;
  if (!(mscale >= 0.0) || !isfinite((float)mscale)) return DDTREE_EINVAL;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  if (scaling == DDTREE_ROPE_YARN && !(original_positions > kTwoPi * beta_slow)) return DDTREE_EINVAL;
  // Pair index at which a pair makes `beta` turns over the original length.
  auto index_of = [&](double beta) {
    return rot_dim * log(original_positions / (beta * kTwoPi)) / (2.0 * log(theta));
  };
  double low = 0.0, span = 1.0;
  if (scaling == DDTREE_ROPE_YARN) {
    low = fmax(floor(index_of(beta_fast)), 0.0);
    const double high = fmin(ceil(index_of(beta_slow)), (double)(rot_dim - 1));
    span = fmax(high - low, 1e-3);
  }
  memset(rope, 0, sizeof(*rope));
  rope->rot_dim = rot_dim;
  rope->interleaved = interleaved;
  rope->mscale = mscale > 0.0 ? (float)mscale : scaling == DDTREE_ROPE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.f;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = pow(theta, -2.0 * i / rot_dim);
    if (scaling == DDTREE_ROPE_LINEAR) f /= factor;
    if (scaling == DDTREE_ROPE_YARN) {
      const double ramp = fmin(fmax((i - low) / span, 0.0), 1.0);
      f = f / factor * ramp + f * (1.0 - ramp);
    }
    rope->turns[i] = (uint64_t)ldexp(f / kTwoPi, 64);  // f <= 1: below a sixth of a turn
  }
  return DDTREE_OK;
}

extern "C" int ddtree_mla_append(int64_t n_tokens, int n_heads, const ddtree_rope_t* rope, const ddtree_bf16_t* kv_new,
                                 int64_t kv_stride, const ddtree_bf16_t* latent_weight, float eps,
                                 const ddtree_bf16_t* q_rope, int64_t q_token_stride, int64_t q_head_stride,
                                 const int32_t* positions, const int32_t* slots, ddtree_bf16_t* kv_pool,
                                 int64_t pool_rows, ddtree_bf16_t* q_out, int64_t q_out_token_stride,
                                 int64_t q_out_head_stride, uint32_t* status, struct CUstream_st* stream) {
  if (n_tokens < 0 || n_tokens > DDTREE_APPEND_MAX_TOKENS || n_heads < 0 || n_heads > DDTREE_MAX_HEADS) return DDTREE_EINVAL;
  if (!rope_ok(rope) || rope->rot_dim != kRope || !(eps >= 0.f) || !isfinite(eps)) return DDTREE_EINVAL;
  if (!row_ok(kv_pool) || pool_rows < 1 || pool_rows > INT32_MAX || !aligned(latent_weight, 16) || !aligned(status, 4))
    return DDTREE_EINVAL;
  if (n_tokens == 0) {  // nothing to read: the tokens' pointers are not looked at
    DevInfo info;
    return device_ok(&info);
  }
  if (!row_ok(kv_new) || !stride_ok(kv_stride, kRow)) return DDTREE_EINVAL;
  if (!positions || !aligned(positions, 4) || !slots || !aligned(slots, 4)) return DDTREE_EINVAL;
  if (n_heads > 0) {
    if (!row_ok(q_rope) || !row_ok(q_out) || !stride_ok(q_token_stride, kRope) || !stride_ok(q_head_stride, kRope) ||
        !stride_ok(q_out_token_stride, kRope) || !stride_ok(q_out_head_stride, kRope))
      return DDTREE_EINVAL;
    if (q_rope == q_out && (q_token_stride != q_out_token_stride || q_head_stride != q_out_head_stride))
      return DDTREE_EINVAL;
  }
  DevInfo info;
  const int rc = device_ok(&info);
  if (rc != DDTREE_OK) return rc;

  MlaAppendArgs a;
  memset(&a, 0, sizeof(a));
  a.kv = kv_new;
  a.weight = latent_weight;
  a.q = q_rope;
  a.positions = positions;
  a.slots = slots;
  a.pool = kv_pool;
  a.q_out = q_out;
  a.status = status;
  a.kv_stride = kv_stride;
  a.q_token = q_token_stride;
  a.q_head = q_head_stride;
  a.o_token = q_out_token_stride;
  a.o_head = q_out_head_stride;
  a.pool_rows = pool_rows;
  a.eps = eps;
  a.n_tokens = (int32_t)n_tokens;
  a.n_heads = n_heads;
  copy_rope(rope, &a.rope);
  if (launch_mla_append(a, info.sms, (cudaStream_t)stream) != cudaSuccess) {
    cudaGetLastError();
    return DDTREE_ELAUNCH;
  }
  return DDTREE_OK;
}

extern "C" int ddtree_draft_append(int64_t n_tokens, int n_heads, const ddtree_draft_cache_t* cache,
                                   const ddtree_rope_t* rope, const void* q, int64_t q_stride, const void* k,
                                   int64_t k_stride, const void* v, int64_t v_stride, const void* q_weight,
                                   const void* k_weight, float eps, const int32_t* positions, const int32_t* slots,
                                   void* q_out, int64_t q_out_stride, uint32_t* status, struct CUstream_st* stream) {
  if (n_tokens < 0 || n_tokens > DDTREE_APPEND_MAX_TOKENS || n_heads < 0 || n_heads > DDTREE_DRAFT_MAX_HEADS)
    return DDTREE_EINVAL;
  if (!draft_cache_ok(cache) || !rope_ok(rope) || rope->rot_dim > cache->head_dim || rope->rot_dim % 16 ||
      !(eps >= 0.f) || !isfinite(eps))
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

  DraftAppendArgs a;
  memset(&a, 0, sizeof(a));
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_weight = static_cast<const uint16_t*>(q_weight);
  a.k_weight = static_cast<const uint16_t*>(k_weight);
  a.positions = positions;
  a.slots = slots;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_cache = static_cast<uint16_t*>(cache->k);
  a.v_cache = static_cast<uint16_t*>(cache->v);
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
  a.page = make_divider(cache->page_size);
  a.dtype = cache->dtype;
  copy_rope(rope, &a.rope);
  if (launch_draft_append(a, info.sms, (cudaStream_t)stream) != cudaSuccess) {
    cudaGetLastError();
    return DDTREE_ELAUNCH;
  }
  return DDTREE_OK;
}
