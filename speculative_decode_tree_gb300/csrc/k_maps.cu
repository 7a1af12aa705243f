// Page-table growth, verify index layout, slots and positions of a decode
// step, from the requests' lengths (include/ddtree_maps.h).
//
// One launch.  Every CTA takes the exclusive sums over the batch (at most 1024
// requests: four per thread) of keys, new tokens and pages to take, into its
// own shared memory: the same integers everywhere, so each CTA reaches the
// all-or-nothing verdict by itself and no CTA waits for another.  The first
// CTAs then write the lists of tokens and pages (a warp per request, so that
// depths come by pointer doubling over the lanes), the others kv_indices: each
// warp a contiguous share of the whole list, eight consecutive entries per lane
// and 32-byte store (four and 16 where every entry is a table entry, page size
// 1: eight requests 4.2 us, by the other form 4.4).  A lane finds its request by
// bisection once and then only walks forward; page and place in the page advance
// by additions.  (Two and four
// steps' table loads in flight together took 27 and 31 us where one takes 24,
// 1024 requests of 21M entries: registers cost more warps than they gain.)
// A page of a request comes from the table below `held` and from the free list
// above, so no thread reads a table entry that this launch writes.
//
// Integer work.  Calls back to back in a graph: one request 2.4 us and eight
// requests of 359,739 entries 4.2 us (a launch and two dependent loads); 1024
// requests of 21.5M entries 23.7 us (0.57 of the measured copy rate), of which the
// 86 MB of writes alone take 12.7.  The rest there is latency: the sums, which
// every CTA takes, some 5 us, and a table load per step of 256 entries.
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

// The pages of one request: from the table below `held`, from the free list
// above.
struct Pages {
  const int32_t* table;  // its row
  const int32_t* fresh;  // such that fresh[k] is page k >= held
  int held;
  __device__ __forceinline__ int operator[](int k) const { return (k < held ? table : fresh)[k]; }
};
__device__ __forceinline__ Pages pages_of(const MapsArgs& a, const Shared& s, int head, int b) {
  Pages p;
  p.held = s.held[b];
  p.table = a.table + (int64_t)s.row[b] * a.table_stride;
  p.fresh = a.free_pages + ((int64_t)head + s.off[b] - p.held);
  return p;
}
// A page's row for a place in it, or -1 (and BAD_INDEX) when it lies outside the pool.
__device__ __forceinline__ int row_of(const MapsArgs& a, int page, int in) {
  if ((uint32_t)page < (uint32_t)a.n_pages) return page * a.page_size + in;
  flag(a, DDTREE_ST_BAD_INDEX);
  return -1;
}

// The first token_ctas CTAs write the token and page lists, the others kv_indices.
template <bool kSinglePage>  // page_size 1: every entry is a table entry
__global__ void __launch_bounds__(kThreads) maps_kernel(const __grid_constant__ MapsArgs a, int token_ctas) {
  __shared__ Shared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = a.batch, ps = a.page_size;
  await_grid();

  // ---- sums over the batch
  const int head = a.held ? __ldg(a.free_head) : 0;
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
      if (P < 0 || L > INT32_MAX || n < 0 || n > a.max_new || row < 0 || row >= a.table_rows || held < 0 || held > a.table_stride) {
        bad = true;
      } else {
        const int pages = L > 0 ? a.page.quotient((int)L - 1) + 1 : 0;
        bad = bad || pages > a.table_stride;
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

  if ((int)blockIdx.x < token_ctas) {
    const int gtid = blockIdx.x * kThreads + tid, threads = token_ctas * kThreads;
    // ---- entries behind the last token (all of them when the call does nothing)
    for (int t = (ok ? total_new : 0) + gtid; t < B * a.max_new; t += threads) {
      a.new_slots[t] = -1;
      a.positions[t] = -1;
      if (a.token_rows) a.token_rows[t] = -1;
    }
    if (!ok) return;

    // ---- new tokens: a warp per request, two nodes per lane
    for (int b = blockIdx.x * kWarps + warp; b < B; b += token_ctas * kWarps) {
      const int t0 = s.nptr[b], n = s.nptr[b + 1] - t0;
      const int P = s.ptr[b + 1] - s.ptr[b] - n;
      const Pages pages = pages_of(a, s, head, b);
      int page[2], number[2], up[2], depth[2];  // up: next ancestor not yet counted, depth: the steps counted
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int i = lane + 32 * r;
        number[r] = a.page.quotient(P + min(i, max(n - 1, 0)));
        page[r] = i < n ? pages[number[r]] : -1;
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
        a.new_slots[t0 + i] = row_of(a, page[r], P + i - number[r] * ps);
        a.positions[t0 + i] = P + depth[r];
        if (a.token_rows) a.token_rows[t0 + i] = s.row[b];
      }
    }

    // ---- pages to take
    for (int64_t e = gtid; e < total_need; e += threads) {
      const int b = request_of(s.off, B, (int)e);
      const int page = __ldg(a.free_pages + head + e);
      a.table[(int64_t)s.row[b] * a.table_stride + s.held[b] + ((int)e - s.off[b])] = page;
      if (page < 0 || page >= a.n_pages) flag(a, DDTREE_ST_BAD_INDEX);
    }
    return;
  }

  // ---- the verify index layout
  if (!ok) return;
  constexpr int kEntries = kSinglePage ? 4 : 8;  // consecutive entries of a lane: one 16- or 32-byte store
  constexpr uint32_t kStep = 32 * kEntries;
  const uint32_t entries = (uint32_t)total;      // below 2^31, so sums with a few steps stay in 32 bits
  const uint32_t warps = (gridDim.x - token_ctas) * kWarps;
  const uint32_t part = ((entries + warps - 1) / warps + kStep - 1) / kStep * kStep;  // whole steps
  const uint64_t part0 = (uint64_t)((blockIdx.x - token_ctas) * kWarps + warp) * part;
  if (part0 + kEntries * lane >= entries) return;
  uint32_t g0 = (uint32_t)part0 + kEntries * lane;
  const uint32_t end = min((uint32_t)part0 + part, entries);
  const bool vec = ((uintptr_t)a.kv_indices & (4 * kEntries - 1)) == 0;
  int b = request_of(s.ptr, B, (int)g0);
  Pages pages = pages_of(a, s, head, b);
  uint32_t first = s.ptr[b], last = s.ptr[b + 1];  // the request's entries
  // k: page of entry g0, in: its place there; a step moves them by whole pages and a rest.
  int k = a.page.quotient((int)(g0 - first)), in = (int)(g0 - first) - k * ps;
  const int step_pages = a.page.quotient((int)kStep), step_in = (int)kStep - step_pages * ps;
  auto store = [&](uint32_t g, const int (&row)[kEntries]) {
    if (vec && g + kEntries <= entries) {
      if constexpr (kSinglePage) {
        *reinterpret_cast<int4*>(a.kv_indices + g) = make_int4(row[0], row[1], row[2], row[3]);
      } else {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(a.kv_indices + g), "r"(row[0]),
                     "r"(row[1]), "r"(row[2]), "r"(row[3]), "r"(row[4]), "r"(row[5]), "r"(row[6]), "r"(row[7])
                     : "memory");
      }
    } else {
#pragma unroll
      for (int e = 0; e < kEntries; ++e)
        if (g + e < entries) a.kv_indices[g + e] = row[e];
    }
  };
  auto forward = [&]() {
    g0 += kStep;
    k += step_pages;
    in += step_in;
    if (in >= ps) {
      in -= ps;
      ++k;
    }
  };
  while (g0 < end) {
    if (g0 >= last) {
      do ++b;  // requests without keys own no entry
      while ((uint32_t)s.ptr[b + 1] <= g0);
      pages = pages_of(a, s, head, b);
      first = s.ptr[b];
      last = s.ptr[b + 1];
      k = a.page.quotient((int)(g0 - first));
      in = (int)(g0 - first) - k * ps;
    }
    if ((kSinglePage || ps >= kEntries) && g0 + kEntries <= last) {
      // All of one request: at most two pages, or four pages of one entry.
      int row[kEntries];
      if constexpr (kSinglePage) {
        int page[kEntries];
#pragma unroll
        for (int e = 0; e < kEntries; ++e) page[e] = pages[k + e];
#pragma unroll
        for (int e = 0; e < kEntries; ++e) row[e] = row_of(a, page[e], 0);
      } else {
        // Rows count on within a page: one product per page, then additions.
        const int left = ps - in;
        const int p0 = pages[k], p1 = left < kEntries ? pages[k + 1] : p0;
        // Without a sign: a page outside the pool may overflow, and is replaced below.
        const uint32_t from = (uint32_t)p0 * (uint32_t)ps + (uint32_t)in, then = (uint32_t)p1 * (uint32_t)ps - (uint32_t)left;
#pragma unroll
        for (int e = 0; e < kEntries; ++e) row[e] = (int)((e < left ? from : then) + (uint32_t)e);
        if (max((uint32_t)p0, (uint32_t)p1) >= (uint32_t)a.n_pages) {
#pragma unroll
          for (int e = 0; e < kEntries; ++e) row[e] = e < left ? row_of(a, p0, in + e) : row_of(a, p1, e - left);
        }
      }
      store(g0, row);
      forward();
      continue;
    }
    // Near a request's end, or short pages: entry by entry.
    int row[kEntries];
    int bb = b, kk = k, ii = in;
    uint32_t stop = last;
    Pages pp = pages;
#pragma unroll
    for (int e = 0; e < kEntries; ++e) {
      row[e] = -1;
      const uint32_t g = g0 + e;
      if (g >= entries) continue;
      if (g >= stop) {
        do ++bb;
        while ((uint32_t)s.ptr[bb + 1] <= g);
        pp = pages_of(a, s, head, bb);
        stop = s.ptr[bb + 1];
        kk = ii = 0;
      }
      row[e] = row_of(a, pp[kk], ii);
      if (++ii == ps) {
        ii = 0;
        ++kk;
      }
    }
    store(g0, row);
    forward();
  }
}

}  // namespace

cudaError_t launch_maps(const MapsArgs& a, int num_sms, cudaStream_t stream) {
  // A warp per request for the lists, one step of 1024 index entries per CTA
  // at least, as many CTAs as an SM holds at most.
  const int64_t tokens = std::min<int64_t>((a.batch + kWarps - 1) / kWarps, num_sms);
  const int64_t index = a.kv_indices ? std::min<int64_t>((a.capacity + 1023) / 1024, (int64_t)num_sms * 5) : 0;
  const unsigned grid = (unsigned)(tokens + index);
  return launch_early(a.page_size == 1 ? maps_kernel<true> : maps_kernel<false>, grid, kThreads, 0, stream, a, (int)tokens);
}

}  // namespace ddtree
