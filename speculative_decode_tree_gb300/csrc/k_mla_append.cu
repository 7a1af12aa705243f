// Latent rows and rotated queries of new tokens (include/ddtree_append.h):
//   pool[slot] = [ norm(latent) * w | R(p) k_rope ],   q_out = R(p) q_rope.
//
// A warp takes a token, or where tokens are few a slice of it: slice 0 has the
// pool row (64 sixteen-byte chunks of latent, two per lane, and the rope part
// on four lanes) and the first query heads, further slices eight heads each
// (four lanes a head, eight pairs a lane).  Each lane computes the sine and
// cosine of one of the 32 pairs and the warp hands them round by shuffles, so
// nothing is staged in shared memory and no warp waits for another.  The loads
// of the row and of the first sixteen heads are in flight together.  The mean
// square is one warp sum over values that stay in registers; every value is
// read once, rounded once and written once: HBM-bound for many tokens, bound by
// two dependent loads for few.  Calls back to back in a graph: 32 tokens x 8
// heads 1.9 us, 512 x 128 4.0 us, 65,521 x 16 65 us (6.45 TB/s, 0.95 of the
// measured copy rate).  One step of heads in flight instead of two took 76 us.
// Slicing: 512 x 128 took 4.7 us with twice as many slices.
#include "rope.cuh"

namespace ddtree {
namespace {

constexpr int kThreads = 128;
constexpr int kHeadsPerStep = 8;
constexpr int kUnroll = 2;  // steps of heads whose loads are in flight together

// Rotates eight pairs: chunk a holds their first elements and chunk b the
// second ones (half layout), or a and b hold whole pairs one after the other.
template <bool kInterleaved>
__device__ __forceinline__ void rotate(uint4& a, uint4& b, const float2 (&cs)[8]) {
  float x[8], y[8];
  unpack8<false>(a, x);
  unpack8<false>(b, y);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float& u = kInterleaved ? (i < 4 ? x[2 * (i & 3)] : y[2 * (i & 3)]) : x[i];
    float& v = kInterleaved ? (i < 4 ? x[2 * (i & 3) + 1] : y[2 * (i & 3) + 1]) : y[i];
    const float r = u * cs[i].x - v * cs[i].y, t = u * cs[i].y + v * cs[i].x;
    u = r;
    v = t;
  }
  a = pack8<false>(x);
  b = pack8<false>(y);
}

template <bool kInterleaved>
__global__ void __launch_bounds__(kThreads) mla_append_kernel(const __grid_constant__ MlaAppendArgs a, int slices,
                                                              int slice_heads) {
  await_grid();
  const int lane = threadIdx.x & 31;
  const int g = lane & 3, sub = lane >> 2;
  const int c0 = kInterleaved ? 2 * g : g, c1 = kInterleaved ? 2 * g + 1 : g + 4;
  const uint64_t freq = a.rope.turns[lane];
  const uint32_t items = (uint32_t)a.n_tokens * (uint32_t)slices;
  const uint32_t stride = gridDim.x * (kThreads / 32);
  for (uint32_t item = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); item < items; item += stride) {
    const uint32_t n = item / (uint32_t)slices;
    const int slice = (int)(item - n * (uint32_t)slices);
    const int64_t token = n;
    const int32_t pos = __ldg(a.positions + n);
    const int64_t slot = __ldg(a.slots + n);
    const bool has_row = slice == 0;  // what the loads below can be issued for without waiting for pos and slot
    uint4 v[2], w[2], r0, r1;
    if (has_row) {
      const uint4* src = reinterpret_cast<const uint4*>(a.kv + token * a.kv_stride);
      v[0] = __ldg(src + lane);
      v[1] = __ldg(src + lane + 32);
      r0 = __ldg(src + kLatent / 8 + c0);  // lanes 4..31 repeat 0..3
      r1 = __ldg(src + kLatent / 8 + c1);
      if (a.weight) {
        w[0] = __ldg(reinterpret_cast<const uint4*>(a.weight) + lane);
        w[1] = __ldg(reinterpret_cast<const uint4*>(a.weight) + lane + 32);
      }
    }
    const int h_begin = slice * slice_heads, h_end = min(h_begin + slice_heads, a.n_heads);
    uint4 q0[kUnroll], q1[kUnroll];
    auto load_heads = [&](int base) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = base + u * kHeadsPerStep + sub;
        q0[u] = q1[u] = make_uint4(0, 0, 0, 0);
        if (h < h_end) {  // plain loads: q_out may be the same buffer
          const uint4* src = reinterpret_cast<const uint4*>(a.q + token * a.q_token + (int64_t)h * a.q_head);
          q0[u] = src[c0];
          q1[u] = src[c1];
        }
      }
    };
    load_heads(h_begin);
    if (pos < 0) {
      if (pos < -1 && has_row && lane == 0 && a.status) atomicOr(a.status, DDTREE_ST_BAD_LENGTH);
      continue;
    }
    const float2 mine = turn(freq, pos, a.rope.mscale);
    float2 cs[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      cs[i] = make_float2(__shfl_sync(0xffffffffu, mine.x, 8 * g + i), __shfl_sync(0xffffffffu, mine.y, 8 * g + i));
    if (has_row && (slot < 0 || slot >= a.pool_rows)) {
      if (slot != -1 && lane == 0 && a.status) atomicOr(a.status, DDTREE_ST_BAD_INDEX);
    } else if (has_row) {
      uint4* dst = reinterpret_cast<uint4*>(a.pool + slot * kRow);
      if (a.weight) {
        float x[2][8], sum = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          unpack8<false>(v[j], x[j]);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum = fmaf(x[j][i], x[j][i], sum);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        const float scale = rsqrtf(sum * (1.f / kLatent) + a.eps);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float y[8];
          unpack8<false>(w[j], y);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[j][i] = x[j][i] * scale * y[i];
          v[j] = pack8<false>(x[j]);
        }
      }
      rotate<kInterleaved>(r0, r1, cs);
      dst[lane] = v[0];
      dst[lane + 32] = v[1];
      if (lane < 4) {
        dst[kLatent / 8 + c0] = r0;
        dst[kLatent / 8 + c1] = r1;
      }
    }
    for (int base = h_begin; base < h_end; base += kHeadsPerStep * kUnroll) {
      if (base != h_begin) load_heads(base);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = base + u * kHeadsPerStep + sub;
        if (h >= h_end) continue;
        rotate<kInterleaved>(q0[u], q1[u], cs);
        uint4* dst = reinterpret_cast<uint4*>(a.q_out + token * a.o_token + (int64_t)h * a.o_head);
        dst[c0] = q0[u];
        dst[c1] = q1[u];
      }
    }
  }
}

}  // namespace

cudaError_t launch_mla_append(const MlaAppendArgs& a, int num_sms, cudaStream_t stream) {
  // A token is one warp's work where tokens fill the SMs with 8 warps each;
  // fewer tokens are cut into slices, down to eight heads.
  const int steps = std::max(1, (a.n_heads + kHeadsPerStep - 1) / kHeadsPerStep);
  const int64_t want = ((int64_t)num_sms * 8 + a.n_tokens - 1) / a.n_tokens;
  const int slice_steps = (int)std::max<int64_t>(1, steps / std::min<int64_t>(want, steps));
  const int slices = (steps + slice_steps - 1) / slice_steps;
  const int64_t blocks = ((int64_t)a.n_tokens * slices + kThreads / 32 - 1) / (kThreads / 32);
  const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)num_sms * 128);
  const int slice_heads = slice_steps * kHeadsPerStep;
  return launch_early(a.rope.interleaved ? mla_append_kernel<true> : mla_append_kernel<false>, grid, kThreads, 0, stream, a,
                      slices, slice_heads);
}

}  // namespace ddtree
