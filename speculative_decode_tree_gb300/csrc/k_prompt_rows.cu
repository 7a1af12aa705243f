// The prompt attention row by row (include/ddtree_prompt.h).
//
// A warp takes a row (a query token and head) and walks its visible keys and no
// others, 32 at a time: a lane has a key for the scores, and columns for the
// sum.  So nothing that a row does not see has a part in it, not even as a
// product with zero.
//
// It runs behind the tensor-core kernel for the items that one has marked, and
// costs a call without any 1 to 2 us, most of them beside the other's end.  A key
// row is read by one lane alone, 16 bytes after 16 bytes, so what bounds it is the
// latency of those loads: a NaN in the last value of 16,384 (16 + 2 heads of 128
// columns), which marks 512 rows, takes 6.0 ms, one in the first value, which marks
// all, 149.  Spreading an item's rows over the CTAs, one for each warp, took the former
// from 98 to 7.  More registers hold more loads (64, 80 and 118: 8.9, 6.0 and 5.4 ms),
// but with 118 the CTAs find room later, where the other kernel ends (200 prompts of 20
// to 30 tokens 31.3 us, with 80 30.7).
#include "prompt_list.cuh"
#include "rope.cuh"
#include "tc_ptx.cuh"

namespace ddtree {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
// A row may have 2^24 keys, and a sum of n numbers one by one is up to n half steps of 32
// bits off where they are alike (262,144 keys: 0.4 to 0.6 %).  In three levels no sum has
// more than 725 terms.
constexpr int kChain = 724;

template <bool kHalf, int kDim>
__global__ void __launch_bounds__(kThreads, 3) prompt_rows_kernel(const __grid_constant__ PromptArgs a) {
  constexpr int kCols = kDim / 32;  // columns of a lane
  __shared__ int scratch[kWarps + 8];
  __shared__ __align__(16) float query[kWarps][kDim];
  __shared__ uint32_t all;
  await_grid();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int items = a.max_items;
  if (blockIdx.x == gridDim.x - 1) {  // this one gathers the items' words
    if (tid == 0) all = 0;
    __syncthreads();
    uint32_t b = 0;
    for (int i = tid; i < items; i += kThreads) b |= a.words[i];
    b &= ~kPromptAgain;
    if (b) atomicOr(&all, b);
    __syncthreads();
    if (tid == 0) *a.status = all;
    return;
  }
  // A unit is a row for each warp of an item.  Thread t looks at every gridDim-th
  // one, from t gridDim on; those of marked items are done one after the other.
  const int ctas = gridDim.x - 1, parts = (a.tile_tokens * a.group + kWarps - 1) / kWarps;
  const int64_t units = (int64_t)items * parts;
  for (int64_t base = blockIdx.x; base < units; base += (int64_t)ctas * kThreads) {
    const int64_t look = base + (int64_t)ctas * tid;
    const bool marked = look < units && (a.words[look / parts] & kPromptAgain);
    if (!__syncthreads_or(marked)) continue;
    for (int slot = 0; slot < kThreads; ++slot) {
      if (!__syncthreads_or(marked && tid == slot)) continue;
      const int64_t unit = base + (int64_t)ctas * slot;
      const int id = (int)(unit / parts), r = (int)(unit - (int64_t)id * parts) * kWarps + warp;
      PromptItem it;
      if (find_prompt_item<kThreads>(a, id / a.n_kv_heads, scratch, it)) continue;
      const int kv = id % a.n_kv_heads;
      const uint16_t* k = a.k + it.k0 * a.k_stride + kv * kDim;
      const uint16_t* v = a.v + it.k0 * a.v_stride + kv * kDim;
      if (r < it.tokens * a.group) {
        const int token = r / a.group, head = kv * a.group + r - token * a.group;
        const int64_t row = it.q0 + token;
        const int pos = it.pos + token;  // below 0: sees nothing
        const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0, first = min(a.n_sinks, lo);
        const int seen = pos < 0 ? 0 : first + pos - lo + 1;
        const uint16_t* q = a.q + row * a.q_stride + head * kDim;
        __syncwarp();
#pragma unroll
        for (int c = 0; c < kCols / 2; ++c) {
          const float2 x = unpack2<kHalf>(reinterpret_cast<const uint32_t*>(q)[c * 32 + lane]);
          query[warp][2 * (c * 32 + lane)] = x.x;
          query[warp][2 * (c * 32 + lane) + 1] = x.y;
        }
        __syncwarp();
        // Sums of 32 keys (`part`), of kChain of those, and of all.
        float o[kCols], chain[kCols], top = -INFINITY, sum = 0.f, chain_sum = 0.f;
#pragma unroll
        for (int c = 0; c < kCols; ++c) o[c] = chain[c] = 0.f;
        for (int base = 0; base < seen; base += 32) {
          const int x = base + lane, j = x < first ? x : x - first + lo;
          float s = -INFINITY;
          if (x < seen) {
            const uint4* key = reinterpret_cast<const uint4*>(k + j * a.k_stride);
            float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
            for (int c = 0; c < kDim / 8; ++c) {
              float y[8];
              unpack8<kHalf>(key[c], y);
#pragma unroll
              for (int e = 0; e < 8; ++e) part[e & 3] = fmaf(y[e], query[warp][8 * c + e], part[e & 3]);
            }
            s = (part[0] + part[1] + part[2] + part[3]) * a.scale_log2;
          }
          float high = s;
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, d));
          high = fmaxf(high, top);
          const float from = high == -INFINITY ? 0.f : high, keep = ptx::ex2_approx(top - from);
          const float p = x < seen ? ptx::ex2_approx(s - from) : 0.f;
          top = high;
          if (keep != 1.f) {  // the same in the whole warp
            sum *= keep;
            chain_sum *= keep;
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
              o[c] *= keep;
              chain[c] *= keep;
            }
          }
          chain_sum += p;
          float part[kCols];
#pragma unroll
          for (int c = 0; c < kCols; ++c) part[c] = 0.f;
          const int n = min(32, seen - base);
          for (int i = 0; i < n; ++i) {
            const float w = __shfl_sync(0xffffffffu, p, i);
            const int jj = __shfl_sync(0xffffffffu, j, i);
            const uint32_t* val = reinterpret_cast<const uint32_t*>(v + jj * a.v_stride);
#pragma unroll
            for (int c = 0; c < kCols / 2; ++c) {
              const float2 y = unpack2<kHalf>(__ldg(val + c * 32 + lane));
              part[2 * c] = fmaf(w, y.x, part[2 * c]);
              part[2 * c + 1] = fmaf(w, y.y, part[2 * c + 1]);
            }
          }
#pragma unroll
          for (int c = 0; c < kCols; ++c) chain[c] += part[c];
          if (base / 32 % kChain == kChain - 1 || base + 32 >= seen) {
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
              o[c] += chain[c];
              chain[c] = 0.f;
            }
            sum += chain_sum;
            chain_sum = 0.f;
          }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        // As in the other kernel: without a key zero, with nothing but scores of -inf 0 / 0.
        const float by = sum == 0.f ? (pos < 0 ? 0.f : NAN) : 1.f / sum;
        uint32_t* out = reinterpret_cast<uint32_t*>(a.out + row * a.out_stride + head * kDim);
#pragma unroll
        for (int c = 0; c < kCols / 2; ++c) out[c * 32 + lane] = pack2<kHalf>(o[2 * c] * by, o[2 * c + 1] * by);
        if (a.lse && lane == 0) a.lse[row * a.n_heads + head] = sum == 0.f ? (pos < 0 ? -INFINITY : NAN) : (top + log2f(sum)) * 0.6931471805599453f;
      }
    }
  }
}

template <bool kHalf>
cudaError_t launch_dim(const PromptArgs& a, int num_sms, cudaStream_t stream) {
  const unsigned grid = (unsigned)std::min<int64_t>(a.max_items, (int64_t)num_sms * 2) + 1;
  return launch_early(a.head_dim == 64    ? prompt_rows_kernel<kHalf, 64>
                      : a.head_dim == 128 ? prompt_rows_kernel<kHalf, 128>
                                          : prompt_rows_kernel<kHalf, 256>,
                      grid, kThreads, 0, stream, a);
}

}  // namespace

cudaError_t launch_prompt_rows(const PromptArgs& a, int num_sms, cudaStream_t stream) {
  return a.dtype == DDTREE_FP16 ? launch_dim<true>(a, num_sms, stream) : launch_dim<false>(a, num_sms, stream);
}

}  // namespace ddtree
