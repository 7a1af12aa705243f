// Causal attention over packed prompts (include/ddtree_prompt.h) on the tensor
// cores.
//
//   S = Q K^T,  P = 2^(scale S - m),  O = sum P V,  l = sum P,  out = O / l
//
// 4 D flops a visible pair and head, and next to nothing to read: the tensor
// pipe is the bound, and everything else has to run beside it.
//
//  - An item is a run of query tokens of one sequence with the heads of one key
//    head: 128 rows (a token's heads next to each other) are one product tile, so
//    a key tile serves the whole group, and short sequences of many heads fill
//    tiles too.  Two tiles (A and B) share every key tile; while the softmax of
//    one works on its scores, the products of the other run: in order A's PV of key
//    tile i, A's QK of i + 1, then B's.  256 columns take one tile, whose scores
//    have two buffers: QK of i + 1 runs beside the softmax of i.
//  - Roles: a warp that loads (TMA boxes of 64 columns, 128-byte swizzle), a warp
//    that issues the products, and four warps for each tile's softmax, a row a
//    thread: no exchange between threads.  S, P (in place of S) and O live in the
//    tensor memory; P is an operand there, and its first half is multiplied while
//    the second is made.
//  - The reference m moves only when a row's maximum has grown by more than 2^8
//    (2^4 for fp16, whose probabilities carry 2^10); O is then scaled in place by
//    the softmax warps.
//  - Key tiles that no row sees are skipped; those that some rows see in part are
//    masked by bits.  What is masked has probability 0, and 0 times a NaN or an
//    infinity in V is a NaN.  Values that no row of the item sees (behind its last
//    token, between sinks and window: other sequences, memory that nobody wrote)
//    become zeros in shared memory.  What is left are values that other rows of the
//    item see: a row whose sum of probabilities is a number and whose result is none
//    marks its item, and a second grid, placed ahead of time, does marked items row by
//    row (k_prompt_rows.cu).  So only prompts that hold such values pay for them, and
//    not for what keys and queries hold: a score that is no number and that a row sees
//    makes all its outputs so.
//  - A CTA goes through many items, one launch's worth of CTAs through all: the loading
//    warp reads the list ahead and hands each item to the others, and loads and first
//    products of the next one run beside this one's stores (a CTA for each item: 64
//    prompts of 1 to 251 tokens 36.3 us, chunks 252; so 33.0 and 237, and with rows
//    that leave as 64-byte pieces 29.1 and 228; by now 25 to 27 and 219 to 233).
//  - Short sequences take one tile a CTA, two CTAs an SM, and two threads for a row,
//    where the plan's buffer has fewer than 1,024 rows (tokens times group) for each of
//    its sequences; how many come is known on the device alone (32 + 8 heads of 128; 200
//    prompts of 20 to 30 tokens 31 us, with two tiles, as in a buffer of 65,536 tokens,
//    40 to 43; 64 of 150 47 and 48).  Long ones want the two tiles (64 of 300 to 500
//    tokens 129 us, with one 154; 16,384 tokens, 16 + 2 heads of 128, 660 and 765).
//  - Waits are bounded (the plan's wait_limit_us; for the next item 2 s, since a warp
//    without rows waits there while others work).  A role whose wait expires sets
//    TIMEOUT and leaves, the softmax warps at the end of their item, to which they go
//    on without waiting; products in flight are waited for before the tensor memory is
//    given back, copies before the CTA ends.
//
// Measured: 16,384 tokens of 16 + 2 heads of 128 columns (1.1 Tflop) 689 to 696 us where
// inputs change, 1.6 Pflop/s, 638 with the same ones again, by the card's power; the
// products alone take 583.  256 columns take 1,560 to 1,590 us (2.2 Tflop; floor 1,093):
// one product tile an SM, with nothing but the next scores beside its softmax.  A pair of
// tiles goes around in 2,600 clocks, of which its products are 2,048: S ready to P
// stored 1,380, and the rest is P to its products to the next S.  With 64 columns the
// products are 1,024 of 2,250, and that chain is the bound (16,384 tokens 473 us).
// With a CTA for each item it took 517, without any arithmetic in the softmax still
// 475, with P in columns of its own, so that the next S is made beside the softmax,
// 560 (the two tiles' softmaxes meet, and one issuing warp's waits are in each
// other's way), with an issuing thread without elections 544 (for the same reason),
// with the maximum found beside the exponentials 532.
#include <cuda.h>
#include <string.h>

#include <atomic>

#include "f32x2.cuh"
#include "prompt_list.cuh"
#include "rope.cuh"
#include "tc_ptx.cuh"

namespace ddtree {
namespace {

using namespace ptx;

struct PromptMaps {
  CUtensorMap q, k, v;
};

// The products cut a sum off where it does not fit into 32 bits, always towards zero:
// 6.3e-9 of it for every key (values of one sign, 2^16 to 2^22 keys), so that a million
// keys in one sum lost 0.7 %.  Where rows may see more than kLongKeys keys, the form
// kLong ends the sum in the tensor memory after every kFoldKeys and joins the parts in
// the workspace, in 32 bits: 1e-4 of a part at most, 2e-4 where the plain form still
// serves, below half a step of an fp16 probability.  The form's other instructions cost
// 1.7 % (16,384 tokens of 16 + 2 heads of 128: 714 us for 702 in turn), hence the plain
// one.  Parts of 4,096, 8,192 and 16,384 keys: 748, 728 and 721 us there.  kMostSms: SMs
// that a plan has room for.
constexpr int kFoldKeys = 16384, kLongKeys = 32768, kMostSms = 160;
// Bounds of waits below this one take the form kPolls, whose waits never suspend a
// thread, since a try may do so for longer than such a bound.
constexpr uint64_t kShortNs = 1000000ull;
constexpr int kPlain = 0, kLong = 1, kPolls = 2;

// kTiles: product tiles of a CTA.  One tile of 64 or 128 columns leaves room for two
// CTAs on an SM: short sequences, where a CTA's start and end are most of its time.
template <int kDim, int kTiles>
struct Config {
  static constexpr bool kSmall = kTiles == 1 && kDim < 256;
  static constexpr int kCtas = kSmall ? 2 : 1;              // per SM
  static constexpr int kKeys = kDim == 256 ? 64 : 128;      // of a key tile
  static constexpr int kSlabs = kDim / 64;                  // of 64 columns
  static constexpr int kQBytes = 128 * kDim * 2;
  static constexpr int kStageBytes = kKeys * kDim * 2;      // a tile of K or of V
  static constexpr int kStages = kDim == 64 ? (kSmall ? 4 : 10) : kSmall ? 2 : 4;
  static constexpr int kSmem = 1024 + kTiles * kQBytes + kStages * kStageBytes;
  // Tensor memory: S of each tile (256 columns: two buffers), O of each tile.
  static constexpr int kBuffers = kDim == 256 ? 2 : 1;      // of S, for each tile
  static constexpr int kColumns = kSmall ? 256 : 512;
  static constexpr int kOCol = kDim == 256 ? 256 : kTiles * kKeys;
  static_assert(kOCol + kTiles * kDim <= kColumns, "tensor memory");
  // Threads of a row.  With two product tiles one is enough, and the softmax warps
  // take registers from the others; few warps are helped by two.
  static constexpr int kSplit = kSmall ? 2 : 1, kMyKeys = kKeys / kSplit;
  static constexpr int kLoadWarp = 4 * kTiles * kSplit, kIssueWarp = kLoadWarp + 1;
  static constexpr int kThreads = 32 * (kTiles == 2 ? kLoadWarp + 4 : kIssueWarp + 1);
  static constexpr int kList = (DDTREE_MAX_BATCH + 1) * 4;  // of sequences
  static constexpr int kFold = kFoldKeys / kKeys;           // key tiles of one sum in the tensor memory
  static constexpr int64_t kFoldBytes = (int64_t)kTiles * 128 * kDim * 4;
};
constexpr int kShortRows = 1024;  // of an average sequence: above
constexpr uint64_t kDrainNs = 2000000000ull;  // for products and copies in flight where the kernel ends

__host__ __device__ constexpr uint32_t product_desc(int n, bool b_mn_major, bool half) {
  return half ? idesc_bf16_f32(128, n, false, b_mn_major) & ~((1u << 7) | (1u << 10)) : idesc_bf16_f32(128, n, false, b_mn_major);
}

__device__ __forceinline__ void load_box(const CUtensorMap* map, uint32_t dst, int col, int head, int row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(col), "r"(head), "r"(row), "r"(smem_u32(bar))
      : "memory");
}

// Four lanes with four pieces of a row each: lane j gets piece j of the four rows.
__device__ __forceinline__ void turn_pieces(uint4 (&c)[4], int lane) {
#pragma unroll
  for (int step = 1; step < 4; step *= 2) {
    const bool upper = lane & step;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & step) continue;
      uint4 &a = c[i], &b = c[i + step];
      const uint4 give = upper ? a : b;
      const uint4 got = make_uint4(__shfl_xor_sync(0xffffffffu, give.x, step), __shfl_xor_sync(0xffffffffu, give.y, step),
                                   __shfl_xor_sync(0xffffffffu, give.z, step), __shfl_xor_sync(0xffffffffu, give.w, step));
      if (upper) a = got;
      else b = got;
    }
  }
}

// Bits 0 .. h of a word of 32.
__device__ __forceinline__ uint32_t bits_to(int h) { return h < 0 ? 0u : h >= 31 ? 0xffffffffu : (2u << h) - 1u; }

// An item with its key tiles: sinks before every row's window, then from the first
// row's window on.
struct Work {
  PromptItem it;
  int id, kv;  // id -1: there are no more items
  int lo_min, sinks, sink_tiles, n_of[2];  // key tiles of each product tile

  template <int kTiles, int kKeys>
  __device__ __forceinline__ void fill(const PromptArgs& a, const PromptItem& item, int number, int tile_tokens) {
    it = item;
    id = number;
    kv = number % a.n_kv_heads;
    lo_min = a.window > 0 ? max(0, it.pos - a.window + 1) : 0;
    sinks = min(a.n_sinks, lo_min);
    sink_tiles = (sinks + kKeys - 1) / kKeys;
    for (int t = 0; t < 2; ++t) {
      const int last = it.pos + min((t + 1) * tile_tokens, it.tokens) - 1;
      n_of[t] = t >= kTiles || t * tile_tokens >= it.tokens || last < 0 ? 0 : sink_tiles + (last - lo_min + kKeys) / kKeys;
    }
  }
  __device__ __forceinline__ int count() const { return max(n_of[0], n_of[1]); }
  template <int kKeys>
  __device__ __forceinline__ int start(int i) const { return i < sink_tiles ? i * kKeys : lo_min + (i - sink_tiles) * kKeys; }
};

template <int kTiles, int kSplit>
struct Shared {
  uint64_t full[10], empty[10];      // stages: landed, used by every tile
  uint64_t item[2], known[2];        // items (even, odd): written, read by every role
  uint64_t queries, asked;           // landed, multiplied by all keys
  uint64_t scores[2];                // S of a tile (256 columns: of a buffer) is complete
  uint64_t weights[2][2];            // 64 keys of P are written, by each half's threads; the first: O is scaled too, by both
  uint64_t products;                 // 256 columns: PV of a key tile is complete
  uint64_t result[2], stored[2];     // O of a tile is complete, read
  uint64_t drained;
  uint64_t pairs[4];                 // what a row's halves have to say is written
  float tops[2][kTiles][2][kSplit == 2 ? 128 : 1];  // of even and odd key tiles, of both halves: the rows' maxima; at the end their sums
  uint32_t base, word;
  int scratch[28];
  Work items[2];
};

template <bool kHalf, int kDim, int kTiles, int kForm>
__global__ void __launch_bounds__(Config<kDim, kTiles>::kThreads, Config<kDim, kTiles>::kCtas)
prompt_kernel(const __grid_constant__ PromptArgs a, const __grid_constant__ PromptMaps maps) {
  using C = Config<kDim, kTiles>;
  constexpr int kSplit = C::kSplit;
  extern __shared__ uint8_t smem[];
  __shared__ Shared<kTiles, kSplit> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  // What needs no data comes before the wait for the stream's last kernel.
  if (warp == C::kLoadWarp) {
    if (elect_one()) {
      for (const CUtensorMap* m : {&maps.q, &maps.k, &maps.v}) asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
    }
    __syncwarp();
    tmem_alloc(&sh.base, C::kColumns);
    tmem_relinquish();
  }
  if (tid == 0) {
    sh.word = 0;
    mbar_init(&sh.queries, 1);
    mbar_init(&sh.asked, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.scores[i], 1);
      for (int h = 0; h < 2; ++h) mbar_init(&sh.weights[i][h], h == 0 ? 4 * kSplit : 4);
      mbar_init(&sh.result[i], 1);
      mbar_init(&sh.stored[i], 4 * kSplit);
      mbar_init(&sh.item[i], 1);
      mbar_init(&sh.known[i], 1 + 4 * kTiles * kSplit);
    }
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&sh.pairs[i], 2);
    mbar_init(&sh.products, 1);
    mbar_init(&sh.drained, 1);
    fence_mbar_init();
  }
  release_grid();
  await_grid();
  tc_fence_before();
  const uint32_t q_at = (smem_u32(smem) + 1023) & ~1023u, ring = q_at + kTiles * C::kQBytes;
  // Items of this CTA: in every second round from the other end, since a sequence's items are longest first.
  auto number = [&](int round) { return (int64_t)round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x); };
  for (int round = tid; (int64_t)round * gridDim.x < a.max_items; round += C::kThreads)
    if (number(round) < a.max_items) a.words[number(round)] = 0;
  int* starts = reinterpret_cast<int*>(smem + (ring - smem_u32(smem)) + C::kStages * C::kStageBytes);
  const int tiles = list_prompt_items<C::kThreads>(a, starts, sh.scratch);
  const bool bad = tiles < 0;
  const int64_t items = (int64_t)tiles * a.n_kv_heads;
  tc_fence_after();
  const uint32_t tmem = sh.base;
  if (bad || number(0) >= items) {
    if (tid == 0 && bad) a.words[blockIdx.x] = DDTREE_ST_BAD_LENGTH;
    if (warp == C::kLoadWarp) tmem_dealloc(tmem, C::kColumns);
    return;
  }
  // The roles start from here together (without it 33.0 us were 35.7 for the short
  // prompts, and 16,384 tokens of 256 columns took 2,030 in place of 1,680).
  __syncthreads();
  const int tile_tokens = a.tile_tokens / kTiles;
  // Whether O starts anew every kFold key tiles, and what it was goes to the workspace.
  const bool folds = kForm == kLong || (kForm == kPolls && a.folds);
  bool late = false;
  auto try_for = [&](uint64_t* bar, int phase) {
    return kForm == kPolls ? mbar_poll(bar, phase & 1, a.wait_ns) : mbar_wait(bar, phase & 1, a.wait_ns);
  };
  auto wait = [&](uint64_t* bar, int phase) {  // by a whole warp
    if (late) return;
    const bool done = try_for(bar, phase);
    if (!__all_sync(0xffffffffu, done)) {
      late = true;
      atomicOr(&sh.word, DDTREE_ST_TIMEOUT);
    }
  };
  // The item of a round, by every role but the one that writes it.  Warps of a tile that
  // an item leaves empty wait here for as long as the item takes, so this wait goes on
  // (2 s at most) as long as no other one has expired.
  auto take = [&](int round, Work& w) {
    if (late) return false;
    bool done = try_for(&sh.item[round & 1], round >> 1);
    if (!__all_sync(0xffffffffu, done)) {
      const uint64_t until = global_timer_ns() + kDrainNs;
      do {
        const bool expired = *reinterpret_cast<volatile uint32_t*>(&sh.word) & DDTREE_ST_TIMEOUT || global_timer_ns() > until;
        if (__any_sync(0xffffffffu, expired)) {
          late = true;
          atomicOr(&sh.word, DDTREE_ST_TIMEOUT);
          return false;
        }
        done = try_for(&sh.item[round & 1], round >> 1);
      } while (!__all_sync(0xffffffffu, done));
    }
    w = sh.items[round & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.known[round & 1]);
    return w.id >= 0;
  };

  if (warp >= C::kLoadWarp) {
    // 384 threads have 168 registers; 128 x 80 and 256 x 208 are fewer.
    if constexpr (kTiles == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == C::kLoadWarp) {
      int n = 0, asked = 0;  // stages filled, items that had queries
      for (int round = 0;; ++round) {
        const bool more = number(round) < items;
        const int id = more ? (int)number(round) : -1;
        Work w = {};
        w.id = -1;
        if (more) w.fill<kTiles, C::kKeys>(a, prompt_item_at(a, starts, id / a.n_kv_heads), id, tile_tokens);
        const PromptItem& it = w.it;
        const int tiles_here = w.count(), present = w.n_of[1] > 0 ? 2 : 1;
        if (round > 1) wait(&sh.known[round & 1], (round >> 1) - 1);
        if (late) break;  // the others' waits for the item expire
        if (lane == 0) {
          sh.items[round & 1] = w;
          mbar_arrive(&sh.item[round & 1]);
        }
        __syncwarp();
        if (!more) break;
        if (tiles_here == 0) continue;
        if (asked > 0) wait(&sh.asked, asked - 1);
        if (late) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&sh.queries, present * C::kSlabs * tile_tokens * a.group * 128);
          for (int t = 0; t < present; ++t)
            for (int s = 0; s < C::kSlabs; ++s)
              load_box(&maps.q, q_at + t * C::kQBytes + s * 16384, 64 * s, w.kv * a.group, it.q0 + t * tile_tokens, &sh.queries);
        }
        __syncwarp();
        ++asked;
        for (int i = 0; i < 2 * tiles_here; ++i, ++n) {  // K of tile 0, V of tile 0, K of tile 1, ...
          const int stage = n % C::kStages;
          if (n >= C::kStages) wait(&sh.empty[stage], n / C::kStages - 1);
          if (late) break;  // a stage that may be on its way is not filled again
          if (elect_one()) {
            mbar_arrive_expect_tx(&sh.full[stage], C::kStageBytes);
            const int row = it.k0 + w.start<C::kKeys>(i >> 1);
#pragma unroll
            for (int s = 0; s < C::kSlabs; ++s)
              load_box(i & 1 ? &maps.v : &maps.k, ring + stage * C::kStageBytes + s * C::kKeys * 128, 64 * s, w.kv, row, &sh.full[stage]);
          }
          __syncwarp();
        }
        if (late) break;
      }
      // Nothing of this may be on its way when the CTA ends.
      if (asked > 0) mbar_wait(&sh.queries, (asked - 1) & 1, kDrainNs);
      for (int i = max(0, n - C::kStages); i < n; ++i) mbar_wait(&sh.full[i % C::kStages], (i / C::kStages) & 1, kDrainNs);
    }
    if (warp == C::kIssueWarp) {
      // ---- products: one warp for both tiles.  With one for each, the tiles' products
      // interleave and their softmaxes meet (16,384 tokens x 16 heads of 128: 1,050 us
      // instead of 750).
      auto stage_of = [&](int n) { return ring + (n % C::kStages) * C::kStageBytes; };
      auto s_of = [&](int t, int g) { return tmem + (C::kBuffers == 2 ? g & 1 : t) * C::kKeys; };
      auto landed = [&](int n) {
        wait(&sh.full[n % C::kStages], n / C::kStages);
        tc_fence_after();
      };
      // By one thread: S of tile t, its g-th key tile; 64 keys of its O += P V.
      auto score = [&](int t, int g, uint32_t k_at) {
#pragma unroll
        for (int s = 0; s < C::kSlabs; ++s)
          mma_ss_x4<2, 2>(s_of(t, g), desc_sw128(q_at + t * C::kQBytes + s * 16384, 16, 1024), desc_sw128(k_at + s * C::kKeys * 128, 16, 1024),
                          product_desc(C::kKeys, false, kHalf), s > 0);
        mma_commit(&sh.scores[C::kBuffers == 2 ? g & 1 : t]);
      };
      auto accumulate = [&](int t, int g, int h, uint32_t v_at, bool more) {
        mma_ts_x4_step<128>(tmem + C::kOCol + t * kDim, s_of(t, g) + 32 * h, desc_sw128(v_at + h * 64 * 128, C::kKeys * 128, 1024),
                            product_desc(kDim, true, kHalf), more);
      };
      auto used = [&](int n) { mma_commit(&sh.empty[n % C::kStages]); };
      int n = 0, asked = 0;                      // stages used, items that had queries
      int before[2] = {0, 0}, had[2] = {0, 0};   // key tiles of product tiles, items with any
      // It leaves where a wait expires: a stage or queries that it gave back without having
      // waited for them would be filled again while they are on their way.
      auto all_items = [&] {
      for (int round = 0;; ++round) {
        Work k;
        if (!take(round, k)) return;
        const PromptItem& it = k.it;
        const int count = k.count(), present = k.n_of[1] > 0 ? 2 : 1;
        if (count == 0) continue;
        wait(&sh.queries, asked);
        landed(n);
        if (late) return;
        if (elect_one()) {
          for (int t = 0; t < present; ++t)
            if (k.n_of[t] > 0) score(t, before[t], stage_of(n));
          used(n);
          if (count == 1) mma_commit(&sh.asked);
        }
        __syncwarp();
        for (int i = 0; i < count; ++i) {
          const int nk = n + 2 * i + 2, nv = n + 2 * i + 1;  // stages of the next K and of this V
          const uint32_t k_at = stage_of(nk), v_at = stage_of(nv);
          const bool more = i + 1 < count;
          if (more) landed(nk);
          if (late) return;
          if (C::kBuffers == 2 && more) {  // the next scores go to the other buffer
            if (elect_one()) {
              score(0, before[0] + i + 1, k_at);
              used(nk);
            }
            __syncwarp();
          }
          landed(nv);
          if (late) return;
          // Values of keys that no row of the item sees become zeros.
          if (!more || i < k.sink_tiles) {
            const int unseen = (i < k.sink_tiles ? k.sinks : it.pos + it.tokens) - k.start<C::kKeys>(i);
#pragma unroll 1
            for (int at = lane * 16; at < (C::kKeys - unseen) * 128; at += 512) {
#pragma unroll
              for (int s = 0; s < C::kSlabs; ++s)
                asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(v_at + (s + 1) * C::kKeys * 128 - 16 - at), "r"(0) : "memory");
            }
            fence_async_smem();
            __syncwarp();
          }
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            if (i >= k.n_of[t]) continue;
            const int g = before[t] + i, w = C::kBuffers == 2 ? g & 1 : t;
            if (i == 0 && had[t] > 0) wait(&sh.stored[t], had[t] - 1);  // O of the item before
#pragma unroll
            for (int h = 0; h < C::kKeys / 64; ++h) {
              wait(&sh.weights[w][h], C::kBuffers == 2 ? g >> 1 : g);
              if (late) return;
              tc_fence_after();
              if (elect_one()) {
                accumulate(t, g, h, v_at, h > 0 || (folds ? i % C::kFold > 0 : i > 0));
                if (h == C::kKeys / 64 - 1) {
                  if (C::kBuffers == 2) mma_commit(&sh.products);
                  if (i + 1 == k.n_of[t]) mma_commit(&sh.result[t]);
                  else if (C::kBuffers == 1) score(t, g + 1, k_at);  // where P was
                }
              }
              __syncwarp();
            }
          }
          if (elect_one()) {
            used(nv);
            if (C::kBuffers == 1 && more) used(nk);
            if (i + 2 == count) mma_commit(&sh.asked);
          }
          __syncwarp();
        }
        n += 2 * count;
        ++asked;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          before[t] += k.n_of[t];
          had[t] += k.n_of[t] > 0;
        }
      }
      };
      all_items();
      // After an expired wait products may be in flight still.
      if (elect_one()) {
        mma_commit(&sh.drained);
        mbar_wait(&sh.drained, 0, kDrainNs);
      }
      __syncwarp();
    }
  } else {
    if constexpr (kTiles == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ---- softmax: a row a thread, or half a row's keys
    const int t = warp / (4 * kSplit), quarter = warp & 3, half = kSplit == 2 ? (warp >> 2) & 1 : 0, row = quarter * 32 + lane;
    constexpr int kMine = kDim / kSplit;  // columns of O of this thread
    const uint32_t my_lane = (uint32_t)(quarter * 32) << 16, o_mem = tmem + C::kOCol + t * kDim + half * kMine + my_lane;
    constexpr float kShift = kHalf ? 10.f : 0.f, kGrowth = kHalf ? 4.f : 8.f;
    const float scale = fmaxf(fabsf(a.scale_log2), 1.4e-45f);  // its sign goes to the scores; zero becomes the least number
    const uint64_t scales = pair(scale, scale);
    // What the other half of a row has to say, once a key tile.
    int turn = 0;
    auto exchange = [&](float mine) {
      if (kSplit == 1) return mine;
      sh.tops[turn & 1][t][half][row] = mine;
      tc_fence_before();  // the second half's P goes where the first half's scores were
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.pairs[quarter]);
      wait(&sh.pairs[quarter], turn);  // bounded, for one of the two may have left after an expired wait
      tc_fence_after();
      return sh.tops[turn++ & 1][t][half ^ 1][row];
    };
    const int row_token = t * tile_tokens + row / a.group, row_head = row % a.group;
    int before = 0, had = 0;  // key tiles of the items before, items with any
    float4* const parts = reinterpret_cast<float4*>(a.folds) + (((int64_t)blockIdx.x * kTiles + t) * kDim + half * kMine) / 4 * 128 + row;
    for (int round = 0;; ++round) {
      Work k;
      if (!take(round, k)) break;
      const PromptItem& it = k.it;
      const int n = k.n_of[t], token = row_token, head = k.kv * a.group + row_head;
      const bool valid = row < tile_tokens * a.group && token < it.tokens;
      // Rows that are none are computed like the last one, and not stored.
      const int pos = it.pos + (valid ? token : it.tokens - 1);
      const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
      float m = -INFINITY, l = 0.f;
      float m_fold = -INFINITY, l_fold = 0.f;  // of what lies in the workspace
      // Key tiles that every row of the warp sees whole start here to there.
      const int lo_most = __reduce_max_sync(0xffffffffu, lo), start_last = __reduce_min_sync(0xffffffffu, pos) - C::kMyKeys + 1;
      for (int i = 0; i < n; ++i) {
        const int g = before + i, buffer = C::kBuffers == 2 ? g & 1 : t;
        wait(&sh.scores[buffer], C::kBuffers == 2 ? g >> 1 : g);
        tc_fence_after();
        // With one buffer these scores came after the last product, which is complete.
        const bool anew = folds && i > 0 && i % C::kFold == 0;
        if (anew) {
          // What O is goes to the workspace, and O starts anew.
          if constexpr (C::kBuffers == 2) {  // as below
            wait(&sh.products, g - 1);
            tc_fence_after();
          }
          const float by = m_fold == -INFINITY ? 0.f : ex2_approx((m_fold - m) * scale);
#pragma unroll 1
          for (int c = 0; c < kMine; c += 16) {
            uint32_t v[16];
            tmem_ld16(o_mem + c, v);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float4* at = parts + (c / 4 + e) * 128;
              float4 u = make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]), __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]));
              if (i > C::kFold) {  // not the first time
                const float4 w = *at;
                u.x += w.x * by; u.y += w.y * by; u.z += w.z * by; u.w += w.w * by;
              }
              *at = u;
            }
          }
          l_fold = l_fold * by + l;
          l = 0.f;
          m_fold = m;
        }
        const uint32_t s_mem = tmem + buffer * C::kKeys + C::kMyKeys * half + my_lane;
        const uint32_t p_mem = tmem + buffer * C::kKeys + C::kMyKeys / 2 * half + my_lane;
        uint32_t x[C::kMyKeys];
        if constexpr (C::kMyKeys == 128) tmem_ld128(s_mem, x);
        else tmem_ld64(s_mem, x);
        if (a.scale_log2 < 0.f) {
#pragma unroll
          for (int c = 0; c < C::kMyKeys; ++c) x[c] ^= 0x80000000u;
        }
        // Columns up to `high`, and of those the ones from `low` on or below `sink`.
        const int start = k.start<C::kKeys>(i) + C::kMyKeys * half;
        if (i < k.sink_tiles || start > start_last || start < lo_most) {
          const int high = min(pos, (i < k.sink_tiles ? k.sinks : it.keys) - 1) - start;
          const int low = i < k.sink_tiles ? 0 : lo - start, sink = a.n_sinks - start;
#pragma unroll
          for (int w = 0; w < C::kMyKeys / 32; ++w) {
            const uint32_t seen = bits_to(high - 32 * w) & (~bits_to(low - 1 - 32 * w) | bits_to(max(sink, 0) - 1 - 32 * w));
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(seen >> c & 1)) x[32 * w + c] = 0xff800000u;  // -inf
          }
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < C::kMyKeys; c += 8) {
#pragma unroll
          for (int e = 0; e < 4; ++e) top[e] = max3(top[e], __uint_as_float(x[c + 2 * e]), __uint_as_float(x[c + 2 * e + 1]));
        }
        float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        most = fmaxf(most, exchange(most));
        bool raised = false;
        float keep = 1.f;
        if (valid && (most - m) * scale > kGrowth) {  // also the first finite maximum
          keep = m == -INFINITY ? 0.f : ex2_approx((m - most) * scale);
          raised = true;
          m = most;
          l *= keep;
        }
        if (i > 0 && !anew && __any_sync(0xffffffffu, raised)) {
          // With one buffer these scores came after the last product, which is complete.
          if constexpr (C::kBuffers == 2) {
            wait(&sh.products, g - 1);
            tc_fence_after();
          }
#pragma unroll 1
          for (int c = 0; c < kMine; c += 32) {
            uint32_t v[32];
            tmem_ld32(o_mem + c, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * keep);
            tmem_st32(o_mem + c, v);
          }
        }
        // The first half's product goes to all columns of O, the second half's among them.
        if (half == 1) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.weights[buffer][0]);
        }
        const float from = m == -INFINITY ? 0.f : kShift - m * scale;
        const uint64_t froms = pair(from, from);
        // A tile's sum first, then the row's: tens of thousands of equal terms one by
        // one would lose four digits.
        uint64_t part[2] = {0, 0};
#pragma unroll
        for (int h = 0; h < C::kMyKeys / 64; ++h) {
          uint32_t p[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float2 y = apart(fma2(pair(__uint_as_float(x[64 * h + 2 * c]), __uint_as_float(x[64 * h + 2 * c + 1])), scales, froms));
            const float u = ex2_approx(y.x), w = ex2_approx(y.y);
            part[c & 1] = add2(part[c & 1], pair(u, w));
            p[c] = pack2<kHalf>(u, w);
          }
          tmem_st32(p_mem + 32 * h, p);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.weights[buffer][half + h]);
        }
        const float2 sums = apart(add2(part[0], part[1]));
        l += sums.x + sums.y;
      }
      const float fold_by = m_fold == -INFINITY ? 0.f : ex2_approx((m_fold - m) * scale);
      if (folds) l += l_fold * fold_by;
      l += kSplit == 1 ? 0.f : exchange(l);
      // ---- the rows
      // A row that sees no key (pos < 0) is zero; with nothing but scores of -inf it is 0 / 0.
      const float by = l == 0.f ? (pos < 0 ? 0.f : NAN) : 1.f / l;
      const int64_t to = it.q0 + token;
      // A lane has a row; where it stores, eight rows of 64 bytes at once, it has a piece of
      // four neighbouring rows (32 rows of 16 bytes at once keep the loads and stores of a
      // whole SM waiting: 64 short prompts 33.0 -> 28.7 us).
      const int64_t out_at = valid ? to * a.out_stride + (int64_t)head * kDim + half * kMine : -1;
      int64_t four[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) four[i] = __shfl_sync(0xffffffffu, out_at, (lane & ~3) + i);
      // O times zero, added up: no number if one of them is none or no end.
      uint64_t none = 0;
      const uint64_t by2 = pair(by, by), zero = pair(0.f, 0.f);
      if (n > 0) {
        wait(&sh.result[t], had);
        tc_fence_after();
      }
#pragma unroll 1
      for (int c = 0; c < kMine; c += 32) {
        uint32_t v[32];
        if (n > 0) {
          tmem_ld32(o_mem + c, v);
          if (c + 32 == kMine) {  // the next item may have it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.stored[t]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0;
        }
        if (folds && n > C::kFold) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 w = parts[(c / 4 + e) * 128];
            v[4 * e] = __float_as_uint(__uint_as_float(v[4 * e]) + w.x * fold_by);
            v[4 * e + 1] = __float_as_uint(__uint_as_float(v[4 * e + 1]) + w.y * fold_by);
            v[4 * e + 2] = __float_as_uint(__uint_as_float(v[4 * e + 2]) + w.z * fold_by);
            v[4 * e + 3] = __float_as_uint(__uint_as_float(v[4 * e + 3]) + w.w * fold_by);
          }
        }
        uint4 piece[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const uint64_t y = pair(__uint_as_float(v[8 * e + 2 * d]), __uint_as_float(v[8 * e + 2 * d + 1]));
            none = fma2(y, zero, none);
            const float2 z = apart(mul2(y, by2));
            w[d] = pack2<kHalf>(z.x, z.y);
          }
          piece[e] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        turn_pieces(piece, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (four[i] >= 0) *reinterpret_cast<uint4*>(a.out + four[i] + c + 8 * (lane & 3)) = piece[i];
      }
      if (valid) {
        if (a.lse && half == 0) a.lse[to * a.n_heads + head] = l == 0.f ? (pos < 0 ? -INFINITY : NAN) : (m * scale - kShift + log2f(l)) * 0.6931471805599453f;
        const float2 both = apart(none);
        // Where l is no number, a score that the row sees is none, and so are all its outputs:
        // masked keys add zeros to l.
        if (l * 0.f == 0.f && !(both.x + both.y == 0.f)) atomicOr(a.words + k.id, kPromptAgain);
      }
      before += n;
      had += n > 0;
    }
    tc_fence_before();
    __syncwarp();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == C::kLoadWarp) tmem_dealloc(tmem, C::kColumns);
  if (tid == 0 && sh.word) atomicOr(a.words + blockIdx.x, sh.word);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                  const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static std::atomic<EncodeTiledFn> fn{nullptr};
  EncodeTiledFn f = fn.load(std::memory_order_acquire);
  if (!f) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      f = reinterpret_cast<EncodeTiledFn>(p);
      fn.store(f, std::memory_order_release);
    } else {
      cudaGetLastError();
    }
  }
  return f;
}

// [rows, heads, kDim] with boxes of 64 columns; rows past the buffer read as zeros.
bool make_map(CUtensorMap* map, const uint16_t* base, int dtype, int dim, int heads, int rows, int64_t stride, int box_heads, int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows}, es[3] = {1, 1, 1};
  return enc(map, dtype == DDTREE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
             const_cast<uint16_t*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kHalf, int kDim, int kTiles, int kForm>
cudaError_t launch_one(const PromptArgs& a, int num_sms, cudaStream_t stream) {
  using C = Config<kDim, kTiles>;
  static_assert(C::kCtas * (C::kSmem + C::kList + sizeof(Shared<kTiles, C::kSplit>) + 1024) <= 228 * 1024 && C::kStages <= 10, "shared memory");
  PromptMaps maps;
  if (!make_map(&maps.q, a.q, a.dtype, kDim, a.n_heads, a.q_rows, a.q_stride, a.group, a.tile_tokens / kTiles) ||
      !make_map(&maps.k, a.k, a.dtype, kDim, a.n_kv_heads, a.k_rows, a.k_stride, 1, C::kKeys) ||
      !make_map(&maps.v, a.v, a.dtype, kDim, a.n_kv_heads, a.k_rows, a.v_stride, 1, C::kKeys))
    return cudaErrorInvalidValue;
  // The shared-memory limit belongs to the kernel on a device: set once on each.
  static std::atomic<uint64_t> have{0};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (device & 63);
  if (!(have.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(prompt_kernel<kHalf, kDim, kTiles, kForm>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem + C::kList);
    if (e != cudaSuccess) return e;
    have.fetch_or(bit, std::memory_order_release);
  }
  const unsigned grid = (unsigned)std::min<int64_t>(a.max_items, (int64_t)std::min(num_sms, kMostSms) * C::kCtas);
  return launch_early(prompt_kernel<kHalf, kDim, kTiles, kForm>, grid, C::kThreads, C::kSmem + (a.batch + 1) * 4, stream, a, maps);
}

template <bool kHalf, int kDim, int kTiles>
cudaError_t launch(const PromptArgs& a, int num_sms, cudaStream_t stream) {
  return a.wait_ns < kShortNs ? launch_one<kHalf, kDim, kTiles, kPolls>(a, num_sms, stream)
         : a.folds            ? launch_one<kHalf, kDim, kTiles, kLong>(a, num_sms, stream)
                              : launch_one<kHalf, kDim, kTiles, kPlain>(a, num_sms, stream);
}

// Whether sequences are short: rows that the buffer has for each.
bool prompt_short(int batch, int q_rows, int group) { return (int64_t)q_rows * group < (int64_t)batch * kShortRows; }

template <bool kHalf>
cudaError_t launch_dim(const PromptArgs& a, int num_sms, cudaStream_t stream) {
  const bool two = a.tile_tokens > 128 / a.group;
  return a.head_dim == 256   ? launch<kHalf, 256, 1>(a, num_sms, stream)
         : a.head_dim == 128 ? (two ? launch<kHalf, 128, 2>(a, num_sms, stream) : launch<kHalf, 128, 1>(a, num_sms, stream))
                             : (two ? launch<kHalf, 64, 2>(a, num_sms, stream) : launch<kHalf, 64, 1>(a, num_sms, stream));
}

}  // namespace

int prompt_tile_tokens(int batch, int q_rows, int group, int head_dim) {
  return 128 / group * (head_dim == 256 || prompt_short(batch, q_rows, group) ? 1 : 2);
}

// Bytes for sums that go on beyond what stays in the tensor memory; 0 where no row sees that many keys.
int64_t prompt_fold_bytes(int k_rows, int head_dim, int group, int window, int n_sinks, int tile_tokens, int64_t max_items) {
  const int64_t keys = window > 0 ? std::min<int64_t>(k_rows, (int64_t)n_sinks + window + tile_tokens) : k_rows;
  if (keys <= kLongKeys) return 0;
  const bool two = tile_tokens > 128 / group;
  auto bytes = [&](auto config) -> int64_t {
    using C = decltype(config);
    return std::min<int64_t>(max_items, kMostSms * C::kCtas) * C::kFoldBytes;
  };
  return head_dim == 256   ? bytes(Config<256, 1>{})
         : head_dim == 128 ? (two ? bytes(Config<128, 2>{}) : bytes(Config<128, 1>{}))
                           : (two ? bytes(Config<64, 2>{}) : bytes(Config<64, 1>{}));
}

cudaError_t launch_prompt(const PromptArgs& a, int num_sms, cudaStream_t stream) {
  const cudaError_t e = a.dtype == DDTREE_FP16 ? launch_dim<true>(a, num_sms, stream) : launch_dim<false>(a, num_sms, stream);
  return e != cudaSuccess ? e : launch_prompt_rows(a, num_sms, stream);
}

}  // namespace ddtree
