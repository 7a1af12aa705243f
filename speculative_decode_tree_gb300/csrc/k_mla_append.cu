// Latent rows and rotated queries of new tokens (include/ddtree_append.h):
//   pool[slot] = [ norm(latent) * w | R(p) k_rope ],   q_out = R(p) q_rope.
//
// One warp per piece of a token: piece 0 is its pool row (64 sixteen-byte
// chunks of latent, two per lane, and the rope part on four lanes), every
// further piece eight query heads (four lanes a head, eight pairs a lane).
// Each lane computes the sine and cosine of one of the 32 pairs and the warp
// hands them round by shuffles, so nothing is staged in shared memory and no
// warp waits for another.  The mean square is one warp sum over values that
// stay in registers; every value is read once, rounded once and written once,
// so the kernel is bound by HBM when there are many tokens and by its two
// dependent loads when there are few.
#include "rope.cuh"

namespace ddtree {
namespace {

constexpr int kThreads = 256;
constexpr int kHeadsPerPiece = 8;

// Rotates the eight pairs of group g (of four): chunk a holds first elements
// and chunk b second ones (half layout), or a and b hold whole pairs in a row.
// cs is the calling lane's own pair; every lane of the warp takes part.
__device__ __forceinline__ void rotate_group(uint4& a, uint4& b, int g, float2 cs, bool interleaved) {
  float x[8], y[8];
  unpack8<false>(a, x);
  unpack8<false>(b, y);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float c = __shfl_sync(0xffffffffu, cs.x, 8 * g + i), s = __shfl_sync(0xffffffffu, cs.y, 8 * g + i);
    float& u = interleaved ? (i < 4 ? x[2 * (i & 3)] : y[2 * (i & 3)]) : x[i];
    float& v = interleaved ? (i < 4 ? x[2 * (i & 3) + 1] : y[2 * (i & 3) + 1]) : y[i];
    const float r = u * c - v * s, t = u * s + v * c;
    u = r;
    v = t;
  }
  a = pack8<false>(x);
  b = pack8<false>(y);
}

template <bool kInterleaved>
__global__ void __launch_bounds__(kThreads) mla_append_kernel(const __grid_constant__ MlaAppendArgs a, int pieces) {
  const int lane = threadIdx.x & 31;
  const uint32_t items = (uint32_t)a.n_tokens * (uint32_t)pieces;
  const uint32_t stride = gridDim.x * (kThreads / 32);
  for (uint32_t item = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); item < items; item += stride) {
    const uint32_t token = item / (uint32_t)pieces;
    const int piece = (int)(item - token * (uint32_t)pieces);
    const int32_t pos = __ldg(a.positions + token);
    if (pos < 0) {
      if (pos < -1 && piece == 0 && lane == 0 && a.status) atomicOr(a.status, DDTREE_ST_BAD_LENGTH);
      continue;
    }
    const int g = lane & 3;
    const int c0 = kInterleaved ? 2 * g : g, c1 = kInterleaved ? 2 * g + 1 : g + 4;
    if (piece == 0) {
      const int64_t slot = __ldg(a.slots + token);
      if (slot < 0 || slot >= a.pool_rows) {
        if (slot != -1 && lane == 0 && a.status) atomicOr(a.status, DDTREE_ST_BAD_INDEX);
        continue;
      }
      const uint4* src = reinterpret_cast<const uint4*>(a.kv + (int64_t)token * a.kv_stride);
      uint4* dst = reinterpret_cast<uint4*>(a.pool + slot * kRow);
      uint4 v[2] = {__ldg(src + lane), __ldg(src + lane + 32)};
      uint4 r0 = __ldg(src + kLatent / 8 + c0), r1 = __ldg(src + kLatent / 8 + c1);  // lanes 4..31 repeat 0..3
      const float2 cs = turn(a.rope.turns[lane], pos, a.rope.mscale);
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
          float w[8];
          unpack8<false>(__ldg(reinterpret_cast<const uint4*>(a.weight) + lane + 32 * j), w);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[j][i] = x[j][i] * scale * w[i];
          v[j] = pack8<false>(x[j]);
        }
      }
      rotate_group(r0, r1, g, cs, kInterleaved);
      dst[lane] = v[0];
      dst[lane + 32] = v[1];
      if (lane < 4) {
        dst[kLatent / 8 + c0] = r0;
        dst[kLatent / 8 + c1] = r1;
      }
    } else {
      const int head = (piece - 1) * kHeadsPerPiece + (lane >> 2);
      const bool have = head < a.n_heads;
      uint4 r0 = make_uint4(0, 0, 0, 0), r1 = r0;
      if (have) {  // plain loads: q_out may be the same buffer
        const uint4* src = reinterpret_cast<const uint4*>(a.q + (int64_t)token * a.q_token + (int64_t)head * a.q_head);
        r0 = src[c0];
        r1 = src[c1];
      }
      const float2 cs = turn(a.rope.turns[lane], pos, a.rope.mscale);
      rotate_group(r0, r1, g, cs, kInterleaved);
      if (have) {
        uint4* dst = reinterpret_cast<uint4*>(a.q_out + (int64_t)token * a.o_token + (int64_t)head * a.o_head);
        dst[c0] = r0;
        dst[c1] = r1;
      }
    }
  }
}

}  // namespace

cudaError_t launch_mla_append(const MlaAppendArgs& a, int num_sms, cudaStream_t stream) {
  if (a.n_tokens == 0) return cudaSuccess;
  const int pieces = 1 + (a.n_heads + kHeadsPerPiece - 1) / kHeadsPerPiece;
  const int64_t blocks = ((int64_t)a.n_tokens * pieces + kThreads / 32 - 1) / (kThreads / 32);
  const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)num_sms * 64);
  if (a.rope.interleaved) mla_append_kernel<true><<<grid, kThreads, 0, stream>>>(a, pieces);
  else mla_append_kernel<false><<<grid, kThreads, 0, stream>>>(a, pieces);
  return cudaGetLastError();
}

}  // namespace ddtree
