// Work items of the prompt attention (include/ddtree_prompt.h): a run of query
// tokens of one sequence and one key head.
#pragma once

#include "common.cuh"

namespace ddtree {

// Rows of an item: `tile_tokens` tokens, token by token the group's heads.
// Items of a sequence come last tokens first, since those see the most keys.
struct PromptItem {
  int q0, tokens;   // first query row of the packed buffer, and how many
  int k0, keys;     // the sequence's keys
  int pos;          // position of the first token: keys - queries + its place
};

// Finds item `tile` of the list (without the key head), by a whole CTA of
// kThreads: 0 found, 1 behind the list's end, 2 the sequences are no good.
// `scratch` holds kThreads / 32 + 8 ints of shared memory.
template <int kThreads>
__device__ __forceinline__ int find_prompt_item(const PromptArgs& a, int tile, int* scratch, PromptItem& item) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* found = scratch + kWarps;
  const int per = (a.batch + kThreads - 1) / kThreads;
  int mine = 0;
  int q_at = 0, q_end = 0, k_at = 0, k_end = 0;  // of the thread's last sequence, its only one where they are few
  bool bad = false;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b >= a.batch) break;
    const int q0 = __ldg(a.q_indptr + b), q1 = __ldg(a.q_indptr + b + 1), k0 = __ldg(a.k_indptr + b), k1 = __ldg(a.k_indptr + b + 1);
    q_at = q0;
    q_end = q1;
    k_at = k0;
    k_end = k1;
    bad |= q0 < 0 || q1 < q0 || q1 > a.q_rows || k0 < 0 || k1 < k0 || k1 > a.k_rows;
    if (!bad) mine += (q1 - q0 + a.tile_tokens - 1) / a.tile_tokens;
  }
  if (tid == 0) found[0] = -1;
  bad = __syncthreads_or(bad);
  if (bad) return 2;
  int inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  int before = inc - mine;
  for (int w = 0; w < warp; ++w) before += scratch[w];
  if (before <= tile && tile < before + mine) {
    int left = tile - before;
    for (int b = tid * per;; ++b) {
      const int q0 = per == 1 ? q_at : __ldg(a.q_indptr + b), q1 = per == 1 ? q_end : __ldg(a.q_indptr + b + 1);
      const int tiles = (q1 - q0 + a.tile_tokens - 1) / a.tile_tokens;
      if (left < tiles) {
        const int first = (tiles - 1 - left) * a.tile_tokens;
        const int k0 = per == 1 ? k_at : __ldg(a.k_indptr + b), k1 = per == 1 ? k_end : __ldg(a.k_indptr + b + 1);
        found[0] = q0 + first;
        found[1] = min(a.tile_tokens, q1 - q0 - first);
        found[2] = k0;
        found[3] = k1 - k0;
        found[4] = k1 - k0 - (q1 - q0) + first;
        break;
      }
      left -= tiles;
    }
  }
  __syncthreads();
  if (found[0] < 0) return 1;
  item.q0 = found[0];
  item.tokens = found[1];
  item.k0 = found[2];
  item.keys = found[3];
  item.pos = found[4];
  return 0;
}

// All items: starts[b] is the number of the first one of sequence b (without the key
// head), starts[batch] that of the whole list, which is returned; -1: the sequences
// are no good.  By a whole CTA; `scratch` as above.
template <int kThreads>
__device__ __forceinline__ int list_prompt_items(const PromptArgs& a, int* starts, int* scratch) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.batch + kThreads - 1) / kThreads;
  int mine = 0;
  bool bad = false;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b >= a.batch) break;
    const int q0 = __ldg(a.q_indptr + b), q1 = __ldg(a.q_indptr + b + 1), k0 = __ldg(a.k_indptr + b), k1 = __ldg(a.k_indptr + b + 1);
    bad |= q0 < 0 || q1 < q0 || q1 > a.q_rows || k0 < 0 || k1 < k0 || k1 > a.k_rows;
    starts[b] = mine;
    if (!bad) mine += (q1 - q0 + a.tile_tokens - 1) / a.tile_tokens;
  }
  int inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) scratch[warp] = inc;
  if (__syncthreads_or(bad)) return -1;
  int before = inc - mine, total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  for (int i = 0; i < per && tid * per + i < a.batch; ++i) starts[tid * per + i] += before;
  if (tid == 0) starts[a.batch] = total;
  __syncthreads();
  return total;
}

// Item `tile` of that list.
__device__ __forceinline__ PromptItem prompt_item_at(const PromptArgs& a, const int* starts, int tile) {
  int b = 0, end = a.batch;  // starts[b] <= tile < starts[end]
  while (end - b > 1) {
    const int mid = (b + end) >> 1;
    if (starts[mid] <= tile) b = mid;
    else end = mid;
  }
  const int q0 = __ldg(a.q_indptr + b), q1 = __ldg(a.q_indptr + b + 1), k0 = __ldg(a.k_indptr + b), k1 = __ldg(a.k_indptr + b + 1);
  const int first = (starts[b + 1] - 1 - tile) * a.tile_tokens;
  PromptItem item;
  item.q0 = q0 + first;
  item.tokens = min(a.tile_tokens, q1 - q0 - first);
  item.k0 = k0;
  item.keys = k1 - k0;
  item.pos = k1 - k0 - (q1 - q0) + first;
  return item;
}

}  // namespace ddtree
