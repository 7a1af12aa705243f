// Page-table growth, verify index layout, slots and positions of a decode
// step, from the requests' lengths (include/ddtree_maps.h).
//
// One launch.  Every CTA takes the exclusive sums over the batch (at most 1024
// requests: four per thread) of keys, new tokens and pages to take, into its
// own shared memory: the same integers everywhere, so each CTA reaches the
// all-or-nothing verdict by itself and no CTA waits for another.  Then the
// CTAs share out three flat lists by element: the pages to take, the new
// tokens (a warp per request, so that depths come by pointer doubling over the
// lanes), and kv_indices, where each thread writes four consecutive entries
// with one 16-byte store and finds its request by bisection of the sums.
// A page of a request comes from the table below `held` and from the free list
// above, so no thread reads a table entry that this launch writes.
//
// Integer work: bounded by the index writes for large batches and by the
// launch and two dependent loads for small ones.
#include "common.cuh"

namespace ddtree {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = DDTREE_MAX_BATCH / kThreads;

struct Shared {
  int32_t ptr[DDTREE_MAX_BATCH + 1];   // exclusive sums of P + n
  int32_t nptr[DDTREE_MAX_BATCH + 1];  // of n
  int32_t off[DDTREE_MAX_BATCH + 1];   // of pages to take
  int32_t held[DDTREE_MAX_BATCH];
  int32_t row[DDTREE_MAX_BATCH];
  long long warp_keys[kWarps], warp_need[kWarps];
  int32_t warp_new[kWarps];
};

__device__ __forceinline__ void flag(const MapsArgs& a, uint32_t bit) {
  if (a.status) atomicOr(a.status, bit);
}

template <typename T>
__device__ __forceinline__ T warp_inclusive(T v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const T o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// The last b with sums[b] <= g, for g < sums[batch].
__device__ __forceinline__ int request_of(const int32_t* sums, int batch, int g) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sums[mid] <= g) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Page k of request b, or -1 (and BAD_INDEX) when it lies outside the pool.
__device__ __forceinline__ int page_of(const MapsArgs& a, const Shared& s, int head, int b, int k) {
  const int page = k < s.held[b] ? a.table[(int64_t)s.row[b] * a.table_stride + k]
                                 : __ldg(a.free_pages + head + s.off[b] + (k - s.held[b]));
  if (page >= 0 && page < a.n_pages) return page;
  flag(a, DDTREE_ST_BAD_INDEX);
  return -1;
}

__global__ void __launch_bounds__(kThreads) maps_kernel(const MapsArgs a) {
  __shared__ Shared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = a.batch, ps = a.page_size;

  // ---- sums over the batch
  long long keys[kPer], need[kPer];
  int fresh[kPer];
  long long keys_sum = 0, need_sum = 0;
  int new_sum = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * kPer + i;
    keys[i] = need[i] = 0;
    fresh[i] = 0;
    if (b < B) {
      const int P = __ldg(a.prefix_lens + b);
      const int n = a.new_lens ? __ldg(a.new_lens + b) : a.max_new;
      const int row = a.table_row ? __ldg(a.table_row + b) : b;
      const int held = a.held ? __ldg(a.held + b) : a.table_stride;
      const long long L = (long long)P + n;
      const long long pages = (L + ps - 1) / ps;
      if (P < 0 || n < 0 || n > a.max_new || row < 0 || row >= a.table_rows || held < 0 || held > a.table_stride ||
          pages > a.table_stride) {
        bad = true;
      } else {
        keys[i] = L;
        fresh[i] = n;
        need[i] = pages > held ? pages - held : 0;
      }
      s.held[b] = held;
      s.row[b] = row;
    }
    keys_sum += keys[i];
    need_sum += need[i];
    new_sum += fresh[i];
  }
  const long long keys_inc = warp_inclusive(keys_sum, lane), need_inc = warp_inclusive(need_sum, lane);
  const int new_inc = warp_inclusive(new_sum, lane);
  if (lane == 31) {
    s.warp_keys[warp] = keys_inc;
    s.warp_need[warp] = need_inc;
    s.warp_new[warp] = new_inc;
  }
  bad = __syncthreads_or(bad);
  long long keys_at = keys_inc - keys_sum, need_at = need_inc - need_sum, total = 0, total_need = 0;
  int new_at = new_inc - new_sum, total_new = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) {
      keys_at += s.warp_keys[w];
      need_at += s.warp_need[w];
      new_at += s.warp_new[w];
    }
    total += s.warp_keys[w];
    total_need += s.warp_need[w];
    total_new += s.warp_new[w];
  }
  const int head = a.held ? __ldg(a.free_head) : 0;
  bad = bad || total > INT32_MAX || (a.kv_indices && total > a.capacity);
  const bool dry = !bad && a.held && (head < 0 || head > a.n_free || total_need > a.n_free - head);
  const bool ok = !bad && !dry;
  if (!ok && blockIdx.x == 0 && tid == 0) flag(a, bad ? DDTREE_ST_BAD_LENGTH : DDTREE_ST_NO_PAGES);
  // 32 bits hold the sums of a call that goes ahead.
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * kPer + i;
    if (b < B) {
      s.ptr[b] = (int32_t)keys_at;
      s.nptr[b] = new_at;
      s.off[b] = (int32_t)need_at;
      keys_at += keys[i];
      new_at += fresh[i];
      need_at += need[i];
      if (blockIdx.x == 0) {
        a.kv_indptr[b] = ok ? s.ptr[b] : 0;
        if (a.new_indptr) a.new_indptr[b] = ok ? s.nptr[b] : 0;
        if (a.held) a.held_out[b] = s.held[b] + (ok ? (int)need[i] : 0);
      }
    }
  }
  if (tid == 0) {
    s.ptr[B] = (int32_t)total;
    s.nptr[B] = total_new;
    s.off[B] = (int32_t)total_need;
    if (blockIdx.x == 0) {
      a.kv_indptr[B] = ok ? (int32_t)total : 0;
      if (a.new_indptr) a.new_indptr[B] = ok ? total_new : 0;
      if (a.held) *a.free_head_out = head + (ok ? (int)total_need : 0);
    }
  }
  __syncthreads();

  const int64_t gtid = (int64_t)blockIdx.x * kThreads + tid;
  const int64_t threads = (int64_t)gridDim.x * kThreads;
  // ---- entries behind the last token (all of them when the call does nothing)
  for (int64_t t = (ok ? total_new : 0) + gtid; t < (int64_t)B * a.max_new; t += threads) {
    a.new_slots[t] = -1;
    a.positions[t] = -1;
    if (a.token_rows) a.token_rows[t] = -1;
  }
  if (!ok) return;

  // ---- pages to take
  for (int64_t e = gtid; e < total_need; e += threads) {
    const int b = request_of(s.off, B, (int)e);
    const int page = __ldg(a.free_pages + head + e);
    a.table[(int64_t)s.row[b] * a.table_stride + s.held[b] + ((int)e - s.off[b])] = page;
    if (page < 0 || page >= a.n_pages) flag(a, DDTREE_ST_BAD_INDEX);
  }

  // ---- new tokens: a warp per request, two nodes per lane
  for (int b = blockIdx.x * kWarps + warp; b < B; b += gridDim.x * kWarps) {
    const int t0 = s.nptr[b], n = s.nptr[b + 1] - t0;
    const int P = s.ptr[b + 1] - s.ptr[b] - n;
    int up[2], depth[2];  // next ancestor not yet counted, and the steps counted
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = lane + 32 * r;
      up[r] = i - 1;
      depth[r] = i;
      if (a.parent) {
        int p = i < n ? __ldg(a.parent + (int64_t)b * a.max_new + i) : -1;
        if (p < -1 || p >= i) {
          flag(a, DDTREE_ST_BAD_PARENT);
          p = -1;
        }
        up[r] = p;
        depth[r] = p >= 0;
      }
    }
    if (a.parent) {
#pragma unroll
      for (int step = 0; step < 6; ++step) {  // ancestors of a 64-node tree: 2^6 steps
        int d[2], u[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int src = up[r] & 31;
          const int d0 = __shfl_sync(0xffffffffu, depth[0], src), d1 = __shfl_sync(0xffffffffu, depth[1], src);
          const int u0 = __shfl_sync(0xffffffffu, up[0], src), u1 = __shfl_sync(0xffffffffu, up[1], src);
          d[r] = up[r] < 32 ? d0 : d1;
          u[r] = up[r] < 32 ? u0 : u1;
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (up[r] >= 0) {
            depth[r] += d[r];
            up[r] = u[r];
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = lane + 32 * r;
      if (i >= n) continue;
      const int page = page_of(a, s, head, b, (P + i) / ps);
      a.new_slots[t0 + i] = page < 0 ? -1 : page * ps + (P + i) % ps;
      a.positions[t0 + i] = P + depth[r];
      if (a.token_rows) a.token_rows[t0 + i] = s.row[b];
    }
  }

  // ---- the verify index layout, four entries per thread
  if (!a.kv_indices) return;
  const bool vec = ((uintptr_t)a.kv_indices & 15) == 0;
  for (int64_t g0 = 4 * gtid; g0 < total; g0 += 4 * threads) {
    int b = request_of(s.ptr, B, (int)g0);
    int end = s.ptr[b + 1];
    unsigned j = (unsigned)((int)g0 - s.ptr[b]);
    unsigned k = j / (unsigned)ps, in = j - k * (unsigned)ps;
    int page = page_of(a, s, head, b, k);
    int out[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      out[e] = page < 0 ? -1 : page * ps + (int)in;
      if (e == 3) break;
      if (g0 + e + 1 >= total) break;
      const int g = (int)(g0 + e + 1);
      if (g >= end) {
        do ++b;  // requests without keys own no entry
        while (s.ptr[b + 1] <= g);
        end = s.ptr[b + 1];
        k = in = 0;
        page = page_of(a, s, head, b, 0);
      } else if (++in == (unsigned)ps) {
        in = 0;
        page = page_of(a, s, head, b, ++k);
      }
    }
    if (vec && g0 + 4 <= total) {
      *reinterpret_cast<int4*>(a.kv_indices + g0) = make_int4(out[0], out[1], out[2], out[3]);
    } else {
      for (int e = 0; e < 4 && g0 + e < total; ++e) a.kv_indices[g0 + e] = out[e];
    }
  }
}

}  // namespace

cudaError_t launch_maps(const MapsArgs& a, int num_sms, cudaStream_t stream) {
  // One CTA per 2048 index entries (two 16-byte stores a thread), up to four
  // per SM; without indices the token lists size the grid.
  const int64_t work = std::max<int64_t>(a.capacity, (int64_t)a.batch * a.max_new * 4);
  const int64_t blocks = std::min<int64_t>((work + 2047) / 2048, (int64_t)num_sms * 4);
  maps_kernel<<<(unsigned)std::max<int64_t>(blocks, 1), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace ddtree
