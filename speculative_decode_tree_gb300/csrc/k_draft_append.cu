// The drafter's new queries, keys and values (include/ddtree_append.h): head
// norms, rotation of the leading columns, cache writes.
//
// A warp takes a token, or a slice of its heads where tokens are few, and
// treats query, key and value heads as one list.  A lane keeps the same 16-byte
// chunk of every head it meets (8, 4, 2 or 1 heads per step for 32 lanes of 8
// columns), so the sines and cosines of its pairs stay in its registers: each
// lane computes a few of the token's pairs and the warp hands them round by
// shuffles once.  A head's mean square is a shuffle sum over its lanes, and in
// the half layout the other element of a pair comes from its lane by shuffle.
// No shared memory, no barrier; kUnroll steps' loads are in flight together.
// Every value is read once, rounded once and written once.  Calls back to back
// in a graph: 8 tokens of 48 heads 3.1 us (launch and two dependent loads);
// 32,749 tokens of 24 64-column heads, interleaved and without norms, 35 us (5.75
// TB/s, 0.85 of the measured copy rate), bound by the memory system: half of the
// cache rows' bytes go out as 128-byte pieces at scattered places, and neither
// more loads in flight (unroll 4 and 6: 36.7 and 35.5 us) nor more warps (unroll
// 2: 35.7) change it.  With norms 40 us, in the half layout 38 and 44.5 (128 and
// 256 columns of the same bytes 47.6 and 49.1): the arithmetic and the exchanges
// between lanes bound those, and 64 registers spill 16 to 24 bytes in the half
// layout.
// The grid holds one wave: 45 us with a CTA per eight tokens.
#include "rope.cuh"

namespace ddtree {
namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 3;

template <bool kHalf, int kDim, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 8) draft_append_kernel(const __grid_constant__ DraftAppendArgs a, int slices,
                                                                int slice_heads) {
  constexpr int kChunks = kDim / 8;              // lanes of a head: 8, 16 or 32
  constexpr int kHeadsPerStep = 32 / kChunks;
  constexpr int kPairsPerLane = kDim / 64;       // pairs a lane computes: dim / 2 over 32 lanes
  constexpr int kTurns = kInterleaved ? 4 : 8;   // pairs with elements in a chunk
  await_grid();
  const int lane = threadIdx.x & 31;
  const int c = lane % kChunks, sub = lane / kChunks;
  const int nq = a.n_heads, nk = a.n_kv_heads, heads = nq + 2 * nk;
  const int pairs = a.rope.rot_dim / 2;
  // Half layout: the chunk that holds the other elements of this chunk's pairs.
  const int half = a.rope.rot_dim / 16;
  const bool turned = 8 * c < a.rope.rot_dim;
  const int other = !turned ? c : c < half ? c + half : c - half;
  const int other_lane = (lane & ~(kChunks - 1)) + other;
  const int pair0 = kInterleaved ? 4 * c : 8 * (c < half ? c : other);
  const bool norms = a.q_weight || a.k_weight;
  const uint4 one = make_uint4(0, 0, 0, 0);
  const uint4 wq = a.q_weight ? __ldg(reinterpret_cast<const uint4*>(a.q_weight) + c) : one;
  const uint4 wk = a.k_weight ? __ldg(reinterpret_cast<const uint4*>(a.k_weight) + c) : one;

  const uint32_t items = (uint32_t)a.n_tokens * (uint32_t)slices;
  const uint32_t stride = gridDim.x * (kThreads / 32);
  for (uint32_t item = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); item < items; item += stride) {
    const uint32_t n = item / (uint32_t)slices;
    const int h_begin = (int)(item - n * (uint32_t)slices) * slice_heads;
    const int h_end = min(h_begin + slice_heads, heads);
    const int64_t token = n;
    const int32_t pos = __ldg(a.positions + n);
    const int32_t slot = __ldg(a.slots + n);
    float2 cs[kTurns];
    const uint16_t *q = a.q + token * a.q_stride, *k = a.k + token * a.k_stride, *v = a.v + token * a.v_stride;
    for (int base = h_begin; base < h_end; base += kHeadsPerStep * kUnroll) {
      uint4 in[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = base + u * kHeadsPerStep + sub;
        const uint16_t* src = h < nq ? q + h * kDim : h < nq + nk ? k + (h - nq) * kDim : v + (h - nq - nk) * kDim;
        in[u] = h < h_end ? reinterpret_cast<const uint4*>(src)[c] : one;  // plain loads: q_out may be q
      }
      if (base == h_begin) {
        if (pos < 0) {
          if (pos < -1 && a.status && h_begin == 0 && lane == 0) atomicOr(a.status, DDTREE_ST_BAD_LENGTH);
          break;
        }
        if (slot < -1 || slot >= a.total_slots) {
          if (a.status && lane == 0) atomicOr(a.status, DDTREE_ST_BAD_INDEX);
        }
        // Pair p is computed by lane p % 32 as its (p / 32)-th.
        float2 mine[kPairsPerLane];
#pragma unroll
        for (int j = 0; j < kPairsPerLane; ++j) {
          const int p = lane + 32 * j;
          mine[j] = p < pairs ? turn(a.rope.turns[p], pos, a.rope.mscale) : make_float2(1.f, 0.f);
        }
#pragma unroll
        for (int t = 0; t < kTurns; ++t) {
          const int p = pair0 + t;
          cs[t] = mine[0];
#pragma unroll
          for (int j = 0; j < kPairsPerLane; ++j) {
            const float x = __shfl_sync(0xffffffffu, mine[j].x, p & 31), y = __shfl_sync(0xffffffffu, mine[j].y, p & 31);
            if (p >> 5 == j) cs[t] = make_float2(x, y);
          }
          // Half layout: a first element is x cos - y sin, a second one x cos + y sin with y its partner.
          if (!kInterleaved && c < half) cs[t].y = -cs[t].y;
        }
      }
      const bool write_kv = slot >= 0 && slot < a.total_slots;
      const int page = write_kv ? a.page.quotient(slot) : 0, off = write_kv ? slot - page * a.page_size : 0;
      const int64_t row = page * a.page_stride + off * a.token_stride;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (base + u * kHeadsPerStep >= h_end) break;  // the same in the whole warp
        const int h = base + u * kHeadsPerStep + sub;
        const bool is_q = h < nq, is_v = h >= nq + nk;
        // Values are copied as they came.  A step of value heads alone leaves the arithmetic out.
        if (base + u * kHeadsPerStep < nq + nk) {
          float x[8];
          unpack8<kHalf>(in[u], x);
          if (norms) {
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
#pragma unroll
            for (int d = kChunks / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            if (is_q ? a.q_weight != nullptr : a.k_weight != nullptr) {
              const float scale = rsqrtf(sum * (1.f / kDim) + a.eps);
              float w[8];
              unpack8<kHalf>(is_q ? wq : wk, w);
#pragma unroll
              for (int j = 0; j < 8; ++j) x[j] = x[j] * scale * w[j];
            }
          }
          if constexpr (kInterleaved) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float e = x[2 * j], o = x[2 * j + 1];
              x[2 * j] = turned ? e * cs[j].x - o * cs[j].y : e;
              x[2 * j + 1] = turned ? e * cs[j].y + o * cs[j].x : o;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float y = __shfl_sync(0xffffffffu, x[j], other_lane);
              if (turned) x[j] = x[j] * cs[j].x + y * cs[j].y;
            }
          }
          if (!is_v) in[u] = pack8<kHalf>(x);
        }
        if (h >= h_end) continue;
        if (is_q) {
          reinterpret_cast<uint4*>(a.q_out + token * a.q_out_stride + h * kDim)[c] = in[u];
        } else if (write_kv) {
          uint16_t* dst = (is_v ? a.v_cache + (h - nq - nk) * a.head_stride : a.k_cache + (h - nq) * a.head_stride) + row;
          reinterpret_cast<uint4*>(dst)[c] = in[u];
        }
      }
    }
  }
}

template <bool kHalf, int kDim>
cudaError_t launch(const DraftAppendArgs& a, int num_sms, cudaStream_t stream) {
  // A token is one warp's work where tokens fill the SMs with 32 warps each;
  // fewer tokens are cut into slices, down to one step of heads.
  constexpr int kHeadsPerStep = 32 / (kDim / 8);
  const int heads = a.n_heads + 2 * a.n_kv_heads;
  const int steps = (heads + kHeadsPerStep - 1) / kHeadsPerStep;
  const int64_t want = ((int64_t)num_sms * 32 + a.n_tokens - 1) / a.n_tokens;
  const int slice_steps = (int)std::max<int64_t>(1, steps / std::min<int64_t>(want, steps));
  const int slices = (steps + slice_steps - 1) / slice_steps;
  const int64_t blocks = ((int64_t)a.n_tokens * slices + kThreads / 32 - 1) / (kThreads / 32);
  const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)num_sms * 8);
  const int slice_heads = slice_steps * kHeadsPerStep;
  return launch_early(a.rope.interleaved ? draft_append_kernel<kHalf, kDim, true> : draft_append_kernel<kHalf, kDim, false>,
                      grid, kThreads, 0, stream, a, slices, slice_heads);
}

}  // namespace

cudaError_t launch_draft_append(const DraftAppendArgs& a, int num_sms, cudaStream_t stream) {
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
