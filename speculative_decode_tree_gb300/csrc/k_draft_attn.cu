// The drafter's attention of one new token per request over its paged cache
// (include/ddtree_draft.h).
//
// One CTA per (token, query head); its warps take the visible keys in turn,
// each with a running maximum and sum in 32 bits, and join at the end.  The
// visible keys are numbered without gaps: the sinks that lie before the
// window, then the window.
#include "rope.cuh"

namespace ddtree {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <bool kHalf, int kDim>
__global__ void __launch_bounds__(kThreads) draft_attn_kernel(const DraftAttnArgs a) {
  constexpr int kPer = kDim / 32;
  __shared__ float acc[kWarps][kDim];
  __shared__ float ms[kWarps], ls[kWarps];
  const int n = blockIdx.x / a.n_heads, h = blockIdx.x - n * a.n_heads, kh = h / a.group;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t* status = reinterpret_cast<uint32_t*>(a.ws);
  const int pos = __ldg(a.positions + n);
  if (pos == -1) return;
  const int row = a.token_rows ? __ldg(a.token_rows + n) : n;
  const bool ok = pos >= 0 && row >= 0 && row < a.table_rows && pos / a.page_size < a.table_stride;
  const int lo = ok && a.window > 0 ? max(0, pos - a.window + 1) : 0;
  const int first = min(a.n_sinks, lo);
  const int64_t seen = ok ? (int64_t)first + pos - lo + 1 : 0;
  if (!ok && threadIdx.x == 0) atomicOr(status, DDTREE_ST_BAD_LENGTH);
  float q[kPer], o[kPer], m = -INFINITY, l = 0.f;
  const uint16_t* qp = a.q + n * a.q_stride + h * kDim;
#pragma unroll
  for (int i = 0; i < kPer / 2; ++i) {
    const float2 p = unpack2<kHalf>(reinterpret_cast<const uint32_t*>(qp)[lane * (kPer / 2) + i]);
    q[2 * i] = p.x;
    q[2 * i + 1] = p.y;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) o[i] = 0.f;
  for (int64_t x = warp; x < seen; x += kWarps) {
    const int j = (int)(x < first ? x : x - first + lo);
    const int page = __ldg(a.table + (int64_t)row * a.table_stride + j / a.page_size);
    if (page < 0 || page >= a.n_pages) {
      if (lane == 0) atomicOr(status, DDTREE_ST_BAD_INDEX);
      continue;
    }
    const int64_t at = page * a.page_stride + (j % a.page_size) * a.token_stride + kh * a.head_stride;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) {
      const float2 p = unpack2<kHalf>(reinterpret_cast<const uint32_t*>(a.k + at)[lane * (kPer / 2) + i]);
      s += q[2 * i] * p.x + q[2 * i + 1] * p.y;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= a.scale_log2;
    const float top = fmaxf(m, s), keep = exp2f(m - top), p = exp2f(s - top);
    m = top;
    l = l * keep + p;
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) {
      const float2 v = unpack2<kHalf>(reinterpret_cast<const uint32_t*>(a.v + at)[lane * (kPer / 2) + i]);
      o[2 * i] = o[2 * i] * keep + p * v.x;
      o[2 * i + 1] = o[2 * i + 1] * keep + p * v.y;
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[warp][lane * kPer + i] = o[i];
  ms[warp] = m;
  ls[warp] = l;
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ms[w]);
  for (int w = 0; w < kWarps; ++w) sum += ms[w] == -INFINITY ? 0.f : ls[w] * exp2f(ms[w] - top);
  for (int c = threadIdx.x; c < kDim / 2; c += kThreads) {
    float x = 0.f, y = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float f = ms[w] == -INFINITY ? 0.f : exp2f(ms[w] - top);
      x += f * acc[w][2 * c];
      y += f * acc[w][2 * c + 1];
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    reinterpret_cast<uint32_t*>(a.out + n * a.out_stride + h * kDim)[c] = pack2<kHalf>(x * inv, y * inv);
  }
  if (threadIdx.x == 0 && a.lse)
    a.lse[(int64_t)n * a.n_heads + h] = sum > 0.f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

int draft_tile_keys(int head_dim) { return head_dim == 256 ? 32 : 64; }

int64_t draft_workspace_bytes(int row_tile, int head_dim, int n_shares) { return 256; }

cudaError_t launch_draft_attention(const DraftAttnArgs& a, cudaStream_t stream) {
  cudaError_t e = cudaMemsetAsync(a.ws, 0, 256, stream);
  if (e != cudaSuccess) return e;
  const unsigned grid = (unsigned)(a.n_tokens * a.n_heads);
#define RUN(H, D) draft_attn_kernel<H, D><<<grid, kThreads, 0, stream>>>(a)
  if (a.dtype == DDTREE_FP16) {
    if (a.head_dim == 64) RUN(true, 64);
    else if (a.head_dim == 128) RUN(true, 128);
    else RUN(true, 256);
  } else {
    if (a.head_dim == 64) RUN(false, 64);
    else if (a.head_dim == 128) RUN(false, 128);
    else RUN(false, 256);
  }
#undef RUN
  return cudaGetLastError();
}

}  // namespace ddtree
