// The drafter's new queries, keys and values (include/ddtree_append.h): head
// norms, rotation of the leading columns, cache writes.
//
// A CTA takes a few tokens and treats all their heads (query, key, value) as
// one list of 16-byte chunks, a chunk per thread and step.  A head's chunks lie
// on neighbouring lanes of one warp, so its mean square is a shuffle sum and
// the second element of a pair in the half layout comes from another lane by
// shuffle.  Sine and cosine are computed once per token and pair into shared
// memory and serve all heads; the loads of the chunks are issued before that.
// Every value is read once, rounded once and written once: HBM-bound for long
// prompts, latency-bound for a decode step.
#include "rope.cuh"

namespace ddtree {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;        // chunks per thread whose loads are in flight together
constexpr int kMaxTokens = 16;    // tokens per CTA

template <bool kHalf, int kDim>
__global__ void __launch_bounds__(kThreads) draft_append_kernel(const __grid_constant__ DraftAppendArgs a,
                                                                int tokens_per_cta) {
  constexpr int kChunks = kDim / 8;  // per head: 8, 16 or 32, a divisor of the warp
  __shared__ float2 table[kMaxTokens][kDim / 2];
  const int lane = threadIdx.x & 31;
  const int heads = a.n_heads + 2 * a.n_kv_heads;
  const int pairs = a.rope.rot_dim / 2;
  const int groups = (a.n_tokens + tokens_per_cta - 1) / tokens_per_cta;
  for (int group = blockIdx.x; group < groups; group += gridDim.x) {
    const int t0 = group * tokens_per_cta;
    const int nt = min(tokens_per_cta, a.n_tokens - t0);
    const int total = nt * heads * kChunks;
    for (int base = 0; base < total; base += kThreads * kUnroll) {
      uint4 v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = base + u * kThreads + (int)threadIdx.x;
        v[u] = make_uint4(0, 0, 0, 0);
        if (i >= total) continue;
        const int c = i % kChunks, hh = i / kChunks, t = hh / heads, h = hh - t * heads;
        const int64_t token = t0 + t;
        const uint16_t* src = h < a.n_heads ? a.q + token * a.q_stride + h * kDim
                              : h < a.n_heads + a.n_kv_heads
                                  ? a.k + token * a.k_stride + (h - a.n_heads) * kDim
                                  : a.v + token * a.v_stride + (h - a.n_heads - a.n_kv_heads) * kDim;
        v[u] = reinterpret_cast<const uint4*>(src)[c];  // plain loads: q_out may be q
      }
      if (base == 0) {
        __syncthreads();  // the last group's rotations are done with the table
        for (int e = threadIdx.x; e < nt * pairs; e += kThreads) {
          const int t = e / pairs, p = e - t * pairs;
          table[t][p] = turn(a.rope.turns[p], max(__ldg(a.positions + t0 + t), 0), a.rope.mscale);
        }
        __syncthreads();
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = base + u * kThreads + (int)threadIdx.x;
        const bool in = i < total;
        const int c = in ? i % kChunks : 0, hh = in ? i / kChunks : 0, t = hh / heads, h = hh - t * heads;
        const bool is_q = h < a.n_heads, is_v = h >= a.n_heads + a.n_kv_heads;
        const uint16_t* weight = is_q ? a.q_weight : is_v ? nullptr : a.k_weight;
        float x[8];
        unpack8<kHalf>(v[u], x);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
#pragma unroll
        for (int d = kChunks / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (weight) {
          float w[8];
          unpack8<kHalf>(__ldg(reinterpret_cast<const uint4*>(weight) + c), w);
          const float scale = rsqrtf(sum * (1.f / kDim) + a.eps);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = x[j] * scale * w[j];
        }
        if (a.rope.interleaved) {
          if (!is_v && 8 * c < a.rope.rot_dim) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 cs = table[t][4 * c + j];
              const float e = x[2 * j], o = x[2 * j + 1];
              x[2 * j] = e * cs.x - o * cs.y;
              x[2 * j + 1] = e * cs.y + o * cs.x;
            }
          }
        } else {
          // The chunk that holds the other elements of this chunk's pairs.
          const int half = a.rope.rot_dim / 16;
          const int other = c < half ? c + half : c < 2 * half ? c - half : c;
          const int src = (lane & ~(kChunks - 1)) + other;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float y = __shfl_sync(0xffffffffu, x[j], src);
            if (!is_v && c < 2 * half) {
              const float2 cs = table[t][8 * (c < half ? c : other) + j];
              x[j] = c < half ? x[j] * cs.x - y * cs.y : y * cs.y + x[j] * cs.x;
            }
          }
        }
        if (!in) continue;
        const int64_t token = t0 + t;
        const int32_t pos = __ldg(a.positions + token);
        if (pos < 0) {
          if (pos < -1 && a.status && h == 0 && c == 0) atomicOr(a.status, DDTREE_ST_BAD_LENGTH);
          continue;
        }
        uint16_t* dst;
        if (is_q) {
          dst = a.q_out + token * a.q_out_stride + h * kDim;
        } else {
          const int64_t slot = __ldg(a.slots + token);
          if (slot < 0 || slot >= a.total_slots) {
            if (slot != -1 && a.status && c == 0) atomicOr(a.status, DDTREE_ST_BAD_INDEX);
            continue;
          }
          const int page = (int)slot / a.page_size, off = (int)slot - page * a.page_size;
          const int kh = h - a.n_heads - (is_v ? a.n_kv_heads : 0);
          dst = (is_v ? a.v_cache : a.k_cache) + page * a.page_stride + off * a.token_stride + kh * a.head_stride;
        }
        // Values are copied as they came.
        reinterpret_cast<uint4*>(dst)[c] = is_v ? v[u] : pack8<kHalf>(x);
      }
    }
  }
}

template <bool kHalf, int kDim>
cudaError_t launch(const DraftAppendArgs& a, int num_sms, cudaStream_t stream) {
  // About one unrolled step of chunks per CTA, but tokens on every SM first.
  const int chunks = (a.n_heads + 2 * a.n_kv_heads) * (kDim / 8);
  int per = std::max(1, std::min(kMaxTokens, kThreads * kUnroll / chunks));
  per = std::max(1, std::min(per, a.n_tokens / num_sms));
  const int64_t blocks = ((int64_t)a.n_tokens + per - 1) / per;
  draft_append_kernel<kHalf, kDim><<<(unsigned)std::min<int64_t>(blocks, (int64_t)num_sms * 64), kThreads, 0, stream>>>(a, per);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_draft_append(const DraftAppendArgs& a, int num_sms, cudaStream_t stream) {
  if (a.n_tokens == 0) return cudaSuccess;
  if (a.dtype == DDTREE_FP16) {
    return a.head_dim == 64    ? launch<true, 64>(a, num_sms, stream)
           : a.head_dim == 128 ? launch<true, 128>(a, num_sms, stream)
                               : launch<true, 256>(a, num_sms, stream);
  }
  return a.head_dim == 64    ? launch<false, 64>(a, num_sms, stream)
         : a.head_dim == 128 ? launch<false, 128>(a, num_sms, stream)
                             : launch<false, 256>(a, num_sms, stream);
}

}  // namespace ddtree
