// The drafter's attention of one new token per request over its paged cache
// (include/ddtree_draft.h).
//
//   s_j = scale <q, k_j>,  out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m)
//
// The work is a stream of keys: 4 D bytes for 4 D flops per query head of the
// group, far below the ridge of some 280 flops a byte, so HBM is the bound.  The
// kernel is built to keep loads in flight on every SM:
//
//  - Equal shares.  The visible keys of a (token, key head) unit are numbered
//    without gaps (the sinks that lie before the window, then the window) and
//    cut into tiles; all units' tiles form one list, and every share takes an
//    equal run of it.  One CTA per share, all resident at once, so every SM
//    streams the same number of bytes whatever the lengths are.  The list exists
//    only as sums over the tokens, which every CTA takes for itself.
//    Up to eight key heads go through the list side by side, one per share:
//    where a token's heads lie next to each other, their shares read the same
//    stretch of memory at the same time (64 columns 192 -> 166 us per GB).
//  - A ring of stages in shared memory, filled by 16-byte cp.async across unit
//    borders: the next unit's first tiles and its queries are under way while
//    the last unit finishes.  A warp of its own runs the page lookups one tile
//    ahead of the copies and leaves row offsets and a validity bit per key in a
//    small ring; a key that is not there is filled with zeros and masked.
//  - The group's query heads are the rows of the matrix instruction (16 rows,
//    padded), so a key row read once serves them all.  Rows are few, and a
//    unit's keys are split over the warps instead, each with its own running
//    maximum and sum in 32 bits; they join through the stage just consumed.
//    This is mma.sync and not tcgen05: with 4 to 16 useful rows of a 128-row
//    tile the tensor pipe is no bound, and the fragments stay in registers.
//    Wide groups take tcgen05 (tensor_tiles, and the rule at Config).
//  - A unit that lies within a share is finished there.  One that crosses into
//    other shares leaves its maximum, sum and unnormalised rows per share (at
//    most two per share), and a second small grid, launched ahead of time with
//    programmatic dependence, joins them in a fixed order.
//
// Measured, calls back to back in a graph, bf16 unless noted: eight requests of
// 1k to 185k tokens, 8 key heads of 128 columns, 205 to 209 us (7.1 TB/s of
// K and V, 1.05 of the measured copy rate); one of 185k with 2 heads of 256
// columns 66.9 us (5.8 TB/s; some 8 us are start, join and launch); 61 fp16
// requests of 511 to 16k, 8 heads of 64 columns, 92 us (6.3 TB/s); a
// window of 2,048 at 65k 7.8 us, a chain of dependent steps (positions, page
// numbers, keys, product, join) with almost no bytes.  64 heads a group stream
// 5.4, 6.2 and 5.3 TB/s at 64, 128 and 256 columns.  Token-granular pages of 64
// columns, 128 bytes at scattered places, stream 5.2 TB/s.
#include <atomic>

#include "rope.cuh"
#include "tc_ptx.cuh"

namespace ddtree {
namespace {

// Keys of a tile and CTAs per SM, by rows and columns.
__host__ __device__ constexpr int keys_of(int row_tile, int dim) {
  return row_tile == 64 ? 8192 / dim : dim == 64 ? 128 : 64;
}
__host__ __device__ constexpr int ctas_of(int row_tile, int dim) { return row_tile == 64 || dim == 256 ? 1 : 2; }

template <int kDim, int kWM>
struct Config {
  // Up to 16 rows, 32 of 64 columns, go through registers, more through the tensor
  // memory (tensor_tiles): in registers every tile of 16 rows loads the keys'
  // fragments for itself, which 64 rows of 128 columns pay with shared memory's
  // whole bandwidth.  us per GB (256 columns: per 537 MB), registers and tensor
  // memory: 64 rows of 64, 128, 256 columns 259, 269, 198 and 197, 172, 101; 24
  // rows 181, 204, 114 and 195, 167, 96.
  static constexpr bool kTensor = kWM == 4;
  static_assert(kWM != 2 || kDim == 64, "see draft_row_tile");
  static constexpr int kKeys = keys_of(16 * kWM, kDim);     // keys of a tile
  // Warps along the rows, the keys and the columns of V.  256 columns are
  // halved between two warps (both take the scores): a whole row's registers
  // would leave too few warps to hide each other's latency.
  static constexpr int kWN = kDim == 256 ? 2 : 1;
  static constexpr int kWK = kTensor ? 2 : kDim == 64 ? 8 / kWM : 4 / kWM;
  static constexpr int kWarps = kTensor ? 12 : kWM * kWN * kWK;
  static constexpr int kThreads = 32 * kWarps;              // that compute
  // One more warp looks the keys up (185k single 70.8 us instead of 84.8 when
  // one of the others did, batch of 61 110 instead of 119).
  static constexpr int kAllThreads = kThreads + (kTensor ? 64 : 32);
  static constexpr int kRows = 16 * kWM;
  static constexpr int kRowBytes = kDim * 2;
  static constexpr int kTileBytes = kKeys * kRowBytes;      // of K, and of V
  static constexpr int kQBytes = kRows * kRowBytes;
  static constexpr int kCtas = ctas_of(16 * kWM, kDim);     // per SM
  static constexpr int kStages = kTensor ? (kDim == 256 ? 4 : 5) : kWM == 1 ? 3 : 2;
  static constexpr int kQSlots = kTensor ? 2 : kStages;     // units whose queries are held
  static constexpr int kRing = kTensor ? 8 : 4;             // offset slots: the tile in use, those in flight, and the next
  static constexpr int kTileRing = kTensor ? 16 : kRing;    // its tiles, begun one ahead of the offsets
  static constexpr int kCopyThreads = kTensor ? 128 : kThreads;
  // Shared memory: probabilities (kTensor), queries, tiles.
  static constexpr int kTileP = kRows * 128 * (kKeys > 64 ? 2 : 1), kPBytes = kTensor ? 2 * kTileP : 0;
  static constexpr int kQAt = kTensor ? kPBytes : kStages * 2 * kTileBytes;  // from the first byte used
  static constexpr int kRingAt = kTensor ? kPBytes + kQSlots * kQBytes : 0;
  static constexpr int kUsed = kPBytes + kQSlots * kQBytes + kStages * 2 * kTileBytes;
  static constexpr int kSmem = (kTensor ? 1024 : 0) + kUsed;
  static_assert(kQAt + kQSlots * kQBytes <= kUsed && kRingAt + kStages * 2 * kTileBytes <= kUsed, "shared memory");
  // The rows of all key parts are joined in the stage that they replace.
  static_assert(kTensor || kWK * kRows * kDim * 4 <= 2 * kTileBytes, "merge buffer");
  static_assert(kRing >= kStages + (kTensor ? 3 : 1), "offset ring");
};

// A unit that goes on from one share to others: where its parts lie.  There is
// a record per unit where units are no more than shares, else one per share,
// for the unit that starts there and goes on; token -1: nothing to join.  (Per
// share alone, CTAs without a unit crowd those with one: window 12.0 us
// instead of 8.0.)
struct Record {
  int32_t token, kv_head, first_share, last_share;
};
__host__ __device__ inline bool by_unit(const DraftAttnArgs& a) { return (int64_t)a.n_tokens * a.n_kv_heads <= a.n_shares; }

// Workspace: status block, per share a status word and a record, then the
// (maximum, sum) pairs and the rows of two partial units per share.
struct Layout {
  int64_t words, records, sums, rows, total;
};
__host__ __device__ inline Layout layout_of(int row_tile, int dim, int shares) {
  Layout l;
  l.words = 256;
  l.records = l.words + ((int64_t)shares * 4 + 255) / 256 * 256;
  l.sums = l.records + ((int64_t)shares * 16 + 255) / 256 * 256;
  l.rows = l.sums + ((int64_t)shares * 2 * row_tile * 8 + 255) / 256 * 256;
  l.total = l.rows + (int64_t)shares * 2 * row_tile * dim * 4;
  return l;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool kHalf>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kHalf) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

// 2^x; results below the normal range become zero.
__device__ __forceinline__ float power2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What a token sees, from its position and table row.
struct Token {
  int pos, row, lo, first, tiles;  // window start, sinks before it, tiles per key head (0: padding)
  int64_t seen;                    // visible keys (0 of a token whose data is bad: one empty tile)
};
__device__ __forceinline__ int row_index(const DraftAttnArgs& a, int n) { return a.token_rows ? __ldg(a.token_rows + n) : n; }
__device__ __forceinline__ Token token_at(const DraftAttnArgs& a, int pos, int row, int tile_keys) {
  Token t;
  t.pos = pos;
  t.row = row;
  const bool ok = t.pos >= 0 && t.row >= 0 && t.row < a.table_rows && a.page.quotient(t.pos) < a.table_stride;
  t.lo = ok && a.window > 0 ? max(0, t.pos - a.window + 1) : 0;
  t.first = min(a.n_sinks, t.lo);
  t.seen = ok ? (int64_t)t.first + t.pos - t.lo + 1 : 0;
  t.tiles = t.pos == -1 ? 0 : ok ? (int)((t.seen + tile_keys - 1) / tile_keys) : 1;
  return t;
}
__device__ __forceinline__ Token token_of(const DraftAttnArgs& a, int n, int tile_keys) {
  return token_at(a, __ldg(a.positions + n), row_index(a, n), tile_keys);
}

// A tile as the copies and the arithmetic need it.
struct Tile {
  int32_t token, kv_head;
  int32_t unit;   // ordinal within the share: its queries' place in the ring
  int32_t flags;
};
enum { kFirst = 1, kLast = 2, kBegun = 4, kGoesOn = 8, kNextLast = 16 };

// ---- 64 rows: scores and sums in tensor memory
//
// Roles: four warps copy, one looks keys up, one issues the products S = Q K^T
// (64 x tile keys) and O += P V (64 x columns), eight take the softmax: four the
// even tiles and four the odd ones, so that one group's exponentials run beside
// the other's loads and maxima.  They hand each row's reference m from tile to
// tile; it moves only when the maximum has grown by more than 2^8 (the rows of O
// are then rescaled in place).  Each group has its own sum, joined where the unit
// ends, and leaves P in shared memory in the cache's type.
// Barriers of stages, tiles and units tie the roles together, so each runs ahead
// as far as its buffers go: copies by the ring's stages, scores by one tile,
// queries by one unit.  What a tile costs now is its copies (32 KB of 16-byte
// copies take an SM some 1,300 of 1,530 cycles at 128 columns), at 64 columns the
// way from scores to product (1,750), at 256 the 18 products (1,740).
// One elected thread of the converged warp issues: with a thread chosen by its
// lane the descriptors go through vector registers, and a product of 16 columns
// of K took 100 cycles to issue instead of 35.
// Waits are bounded (the plan's wait_limit_us): a warp whose wait expires sets
// TIMEOUT and goes on without waiting for copies and products, but meets every
// named barrier, each once a tile and in order, so that all warps come to the end:
//  - P is handed over at four of them in turn (tile & 3).  A warp arrives without
//    waiting there and runs ahead; from an expired wait on it waits there, at a
//    barrier whose last use was over before its tile's scores were issued.  With
//    two in turn it could arrive for the next tile before a slower warp had
//    arrived for this one, and the count would never come out again.
//  - Tiles that other warps take from it may not have been looked up yet; their
//    places hold a valid token from the start, so nothing is read or written out of
//    range.  A softmax warp takes each for a unit's end and leaves its rows in the
//    workspace: what a tile owes to the next one is then the same for every tile.
struct TensorShared {
  // Barriers.  Of a stage: copies landed, O of its tile complete.  Of even and odd
  // tiles: S complete.  Of even and odd units: the last S with their queries complete.
  uint64_t full[5], values[5], scores[2], queries[2];
  uint32_t base;                  // tensor memory
};
constexpr int kAllocWarp = 3, kIssueWarp = 13;
// Named barriers: 0 of all warps, 1 of the copies, eight for the reference of a
// quarter of the rows (from even to odd tiles and back), four for P.
constexpr int kReferenceBarrier = 2, kPBarrier = 10;
constexpr uint64_t kDrainNs = 2000000000ull;  // for products in flight where the kernel ends
// Bounds below this one have a kernel of their own that polls (kShort): a try may
// suspend a warp for longer, and polls beside the tries make the kernel's code so
// long that 64 rows of 64 columns took 309 us per GB instead of 223.
constexpr uint64_t kShortNs = 1000000ull;
// Columns: two S at 0, O behind; a power of two.
__host__ __device__ constexpr int o_col(int dim) { return dim == 128 ? 128 : 256; }
__host__ __device__ constexpr int tmem_cols(int dim) { return dim == 128 ? 256 : 512; }
// Instruction descriptor: 32-bit sums, A and B both fp16 or both bf16, A K-major.
__host__ __device__ constexpr uint32_t product_desc(int n, bool b_mn_major, bool half) {
  return half ? ptx::idesc_bf16_f32(64, n, false, b_mn_major) & ~((1u << 7) | (1u << 10))
              : ptx::idesc_bf16_f32(64, n, false, b_mn_major);
}

// Warps 0 to 7 take the softmax, 8 to 11 copy.
__device__ __forceinline__ bool copies_tiles(int warp) { return (warp & ~3) == 8; }

// The copying warps and the lookup warp.
__device__ __forceinline__ void copies_barrier() { asm volatile("bar.sync 1, 160;" ::: "memory"); }

template <bool kHalf, int kDim, bool kShort, typename Copies, typename Queries>
__device__ __forceinline__ void tensor_tiles(const DraftAttnArgs& a, const Layout& ws, TensorShared& sh, uint32_t p_at,
                                             uint32_t q_ring, uint32_t ring, const Tile* tiles,
                                             const uint32_t (*there)[Config<kDim, 4>::kKeys / 32], float* reference, float2* others,
                                             uint32_t* bits, int count, int share, Copies& start_copies, Queries& start_queries) {
  using namespace ptx;
  using C = Config<kDim, 4>;
  constexpr int kBlocks = C::kKeys / 8;  // of eight keys
  constexpr int kSlab = C::kKeys * 128, kRowSlab = 64 * 128;  // 64 columns of a tile, and of 64 rows
  constexpr float kShift = kHalf ? 10.f : 0.f;
  constexpr float kGrowth = kHalf ? 4.f : 8.f;  // fp16: 2^(10 + 4) is the largest probability
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  tc_fence_after();  // the base was written before the last barrier
  const uint32_t s_mem = sh.base, o_mem = sh.base + o_col(kDim);
  bool late = false;
  auto wait = [&](uint64_t* bar, int phase) {  // by a whole warp
    if (late) return;
    const bool done = kShort ? mbar_poll(bar, phase & 1, a.wait_ns) : mbar_wait(bar, phase & 1, a.wait_ns);
    if (!__all_sync(0xffffffffu, done)) {
      late = true;
      atomicOr(bits, DDTREE_ST_TIMEOUT);
    }
  };
  auto wait_values = [&](int i) { wait(&sh.values[i % C::kStages], i / C::kStages); };
  auto stage_of = [&](int i) { return ring + (i % C::kStages) * 2 * C::kTileBytes; };

  if (copies_tiles(warp)) {
    for (int i = 0; i < count; ++i) {
      __syncwarp();
      copies_barrier();  // the tile's keys are looked up
      if (i >= C::kStages) wait_values(i - C::kStages);
      const Tile t = tiles[i % C::kTileRing];
      if (t.flags & kFirst) {
        if (t.unit >= 2) wait(&sh.queries[t.unit & 1], t.unit / 2 - 1);
        start_queries(i);
      }
      start_copies(i);
      cp_async_mbar_arrive(&sh.full[i % C::kStages]);
      if ((threadIdx.x & 127) == 0) mbar_arrive(&sh.full[i % C::kStages]);  // what the lookup wrote goes along
    }
    return;
  }

  if (warp == kIssueWarp) {
    auto score = [&](int i) {
      wait(&sh.full[i % C::kStages], i / C::kStages);
      fence_async_smem();  // what the copies wrote, before the tensor core reads it
      tc_fence_after();
      if (elect_one()) {
        const Tile t = tiles[i % C::kTileRing];
        const uint32_t q_at = q_ring + (t.unit % C::kQSlots) * C::kQBytes, k_at = stage_of(i);
#pragma unroll
        for (int c = 0; c < kDim / 64; ++c)
          mma_ss_x4<2, 2>(s_mem + (i & 1) * C::kKeys, desc_sw128(q_at + c * kRowSlab, 16, 1024),
                          desc_sw128(k_at + c * kSlab, 16, 1024), product_desc(C::kKeys, false, kHalf), c > 0);
        mma_commit(&sh.scores[i & 1]);
        if (t.flags & kLast) mma_commit(&sh.queries[t.unit & 1]);
      }
      __syncwarp();
    };
    score(0);
    for (int i = 0; i < count; ++i) {
      if (i + 1 < count) score(i + 1);
      asm volatile("bar.sync %0, 160;" ::"r"(kPBarrier + (i & 3)) : "memory");  // P is written and O rescaled
      tc_fence_after();
      if (elect_one()) {
        const uint32_t p_tile = p_at + (i & 1) * C::kTileP, v_at = stage_of(i) + C::kTileBytes;
        const bool more = !(tiles[i % C::kTileRing].flags & kFirst);
        if constexpr (C::kKeys >= 64) {
#pragma unroll
          for (int c = 0; c < C::kKeys / 64; ++c)
            mma_ss_x4<2, 128>(o_mem, desc_sw128(p_tile + c * kRowSlab, 16, 1024), desc_sw128(v_at + c * 64 * 128, kSlab, 1024),
                              product_desc(kDim, true, kHalf), c > 0 || more);
        } else {
          mma_ss_x2<2, 128>(o_mem, desc_sw128(p_tile, 16, 1024), desc_sw128(v_at, kSlab, 1024), product_desc(kDim, true, kHalf),
                            more);
        }
        mma_commit(&sh.values[i % C::kStages]);
      }
      __syncwarp();
    }
    // Nothing is in flight once the softmax warps are through (the last tile
    // ends a unit); after an expired wait, give what is a last chance.
    if (elect_one()) {
      __shared__ uint64_t drained;
      mbar_init(&drained, 1);
      fence_mbar_init();
      mma_commit(&drained);
      mbar_wait(&drained, 0, kDrainNs);
    }
    return;
  }

  // Row 16 w + r of a product with 64 rows is lane 32 w + r of the tensor memory.
  // A thread has rows row and row + 8, keys (columns) 2 quad and 2 quad + 1 of every eight.
  const int quarter = warp & 3, row = quarter * 16 + (lane >> 2), quad = lane & 3;
  const int mine = warp >> 2;  // even tiles or odd ones
  const uint32_t my_lane = (uint32_t)(quarter * 32) << 16;
  const float scale = fmaxf(fabsf(a.scale_log2), 1.4e-45f);  // as for fewer rows
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};  // as of this group's last tile
  int unit = -1;
  for (int i = mine; i < count; i += 2) {
    const int slot = i % C::kRing;
    wait(&sh.scores[i & 1], i >> 1);
    tc_fence_after();
    Tile t = tiles[i % C::kTileRing];
    if (late) t.flags = kLast | kGoesOn;  // the lookup may not have been here
    uint32_t x[4 * kBlocks];
    const uint32_t x_mem = s_mem + my_lane + (i & 1) * C::kKeys;
    if constexpr (kBlocks == 4) tmem_ld_frag32(x_mem, x);
    else
#pragma unroll
      for (int c = 0; c < kBlocks / 8; ++c) tmem_ld_frag64(x_mem + 64 * c, reinterpret_cast<uint32_t(&)[32]>(x[32 * c]));
    if (a.scale_log2 < 0.f) {
#pragma unroll
      for (int k = 0; k < 4 * kBlocks; ++k) x[k] ^= 0x80000000u;
    }
#pragma unroll
    for (int w = 0; w < kBlocks / 4; ++w) {
      const uint32_t mask = there[slot][w];
      if (mask != 0xffffffffu) {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (!((mask >> (8 * (k >> 2) + 2 * quad + (k & 1))) & 1)) x[16 * w + k] = 0xff800000u;  // -inf
      }
    }
    float top[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float high[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < kBlocks; ++j) {
        high[0] = fmaxf(high[0], __uint_as_float(x[4 * j + 2 * h]));
        high[1] = fmaxf(high[1], __uint_as_float(x[4 * j + 2 * h + 1]));
      }
      top[h] = fmaxf(high[0], high[1]);
      top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
      top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
    }
    // The reference goes from tile to tile, and so from group to group; where a
    // unit ends, after its rows were read: the next tile's product writes over them.
    if (i > 0) asm volatile("bar.sync %0, 64;" ::"r"(kReferenceBarrier + 4 - 4 * mine + quarter) : "memory");
    bool raised = false;
    float keep[2], before[2] = {-INFINITY, -INFINITY};
    if (!(t.flags & kFirst)) {
      before[0] = reference[row];
      before[1] = reference[row + 8];
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float now = before[h];
      keep[h] = 1.f;
      if ((top[h] - now) * scale > kGrowth) {  // also the first finite maximum
        keep[h] = now == -INFINITY ? 0.f : power2((now - top[h]) * scale);
        raised = true;
        now = top[h];
      }
      if (unit != t.unit) l[h] = 0.f;
      else if (m[h] != now) l[h] *= m[h] == -INFINITY ? 0.f : power2((m[h] - now) * scale);
      m[h] = now;
      if (quad == 0) reference[row + 8 * h] = now;
    }
    unit = t.unit;
    __syncwarp();
    const bool unit_ends = t.flags & kLast;
    if (!unit_ends) asm volatile("bar.arrive %0, 64;" ::"r"(kReferenceBarrier + 4 * mine + quarter) : "memory");
    if (!(t.flags & kFirst) && __any_sync(0xffffffffu, raised)) {
      wait_values(i - 1);  // the rows of O are complete
      tc_fence_after();
      uint32_t v[16];
#pragma unroll 1
      for (int c = 0; c < kDim; c += 32) {
        tmem_ld_frag32(o_mem + my_lane + c, v);
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * keep[(e >> 1) & 1]);
        tmem_st_frag32(o_mem + my_lane + c, v);
      }
      tmem_st_wait();
    }
    if (i > 1) wait_values(i - 2);  // these probabilities' place is free
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float base = m[h] == -INFINITY ? 0.f : kShift - m[h] * scale;
      const uint32_t p_row = p_at + mine * C::kTileP + (row + 8 * h) * 128 + 4 * quad;
      float sums[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kBlocks; ++j) {
        const float u = power2(fmaf(__uint_as_float(x[4 * j + 2 * h]), scale, base));
        const float w = power2(fmaf(__uint_as_float(x[4 * j + 2 * h + 1]), scale, base));
        sums[j & 1] += u + w;
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(p_row + (j >> 3) * kRowSlab + (((j & 7) ^ (row & 7)) << 4)),
                     "r"(pack2<kHalf>(u, w))
                     : "memory");
      }
      l[h] += sums[0] + sums[1];
    }
    float total[2] = {l[0], l[1]};
    if (t.flags & (kLast | kNextLast)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        total[h] += __shfl_xor_sync(0xffffffffu, total[h], 1);
        total[h] += __shfl_xor_sync(0xffffffffu, total[h], 2);
        // For the group that ends the unit: this one's sum and its reference.
        if (!unit_ends && quad == 0) others[row + 8 * h] = make_float2(total[h], m[h]);
      }
    }
    fence_async_smem();
    tc_fence_before();
    __syncwarp();
    if (late) asm volatile("bar.sync %0, 160;" ::"r"(kPBarrier + (i & 3)) : "memory");
    else asm volatile("bar.arrive %0, 160;" ::"r"(kPBarrier + (i & 3)) : "memory");
    if (!unit_ends) continue;

    // ---- the unit ends here; the product before this tile's came after the other group's sums
    wait_values(i);
    tc_fence_after();
    const bool whole = !(t.flags & (kBegun | kGoesOn));
    const int64_t part = 2 * share + (t.flags & kBegun ? 0 : 1);
    const int head = t.kv_head * a.group + row;
    float inv[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (!(t.flags & kFirst)) {
        const float2 other = others[row + 8 * h];
        if (other.x != 0.f) total[h] += other.x * power2((other.y - m[h]) * scale);
      }
      inv[h] = total[h] == 0.f ? 0.f : 1.f / total[h];
    }
    uint16_t* out = a.out + t.token * a.out_stride + (int64_t)head * kDim + 2 * quad;
    float* rows = reinterpret_cast<float*>(a.ws + ws.rows) + (part * C::kRows + row) * kDim + 2 * quad;
#pragma unroll 1
    for (int c = 0; c < kDim; c += 32) {
      uint32_t v[16];
      tmem_ld_frag32(o_mem + my_lane + c, v);  // the whole warp; the rows that count are stored
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (row + 8 * h < a.group) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float u = __uint_as_float(v[4 * j + 2 * h]), w = __uint_as_float(v[4 * j + 2 * h + 1]);
            if (whole) *reinterpret_cast<uint32_t*>(out + 8 * h * kDim + c + 8 * j) = pack2<kHalf>(u * inv[h], w * inv[h]);
            else *reinterpret_cast<float2*>(rows + 8 * h * kDim + c + 8 * j) = make_float2(u, w);
          }
        }
      }
      __syncwarp();
    }
    tc_fence_before();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (row + 8 * h < a.group && quad == 0) {
        const float top = m[h] == -INFINITY ? m[h] : m[h] * scale;
        if (!whole) reinterpret_cast<float2*>(a.ws + ws.sums)[part * C::kRows + row + 8 * h] = make_float2(top, total[h]);
        else if (a.lse)
          a.lse[(int64_t)t.token * a.n_heads + head + 8 * h] =
              total[h] == 0.f ? -INFINITY : (top - kShift + log2f(total[h])) * 0.6931471805599453f;
      }
    }
    __syncwarp();
    if (i + 1 < count) asm volatile("bar.arrive %0, 64;" ::"r"(kReferenceBarrier + 4 * mine + quarter) : "memory");
  }
  tc_fence_before();
}

template <bool kHalf, int kDim, int kWM, bool kShort>
__global__ void __launch_bounds__(Config<kDim, kWM>::kAllThreads, Config<kDim, kWM>::kCtas)
draft_attn_kernel(const __grid_constant__ DraftAttnArgs a) {
  using C = Config<kDim, kWM>;
  constexpr int kThreads = C::kThreads, kWarps = C::kWarps;  // without the lookup warp
  constexpr int kChunks = kDim / 8;  // 16-byte chunks of a row
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t offsets[C::kRing][C::kKeys];   // element offset of a key's row
  __shared__ uint32_t there[C::kRing][C::kKeys / 32];  // a bit per key that exists
  __shared__ Tile tiles[C::kTileRing];
  __shared__ __align__(8) float top_s[C::kWK][C::kRows], sum_s[C::kWK][C::kRows];  // kTensor: one maximum, one (sum, maximum)
  __shared__ int64_t warp_sum[C::kAllThreads / 32];
  __shared__ int start_token;
  __shared__ int64_t start_at;
  __shared__ uint32_t bits;
  __shared__ TensorShared tensor;  // of the tensor form only

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int share = blockIdx.x, range = share >> a.bundle_log2, sub = share - (range << a.bundle_log2);
  const int bundles = a.n_kv_heads >> a.bundle_log2;
  const Layout ws = layout_of(C::kRows, kDim, a.n_shares);
  Record* records = reinterpret_cast<Record*>(a.ws + ws.records);
  uint32_t* words = reinterpret_cast<uint32_t*>(a.ws + ws.words);
  release_grid();
  await_grid();

  // ---- the list of tiles: sums over the tokens, a run of tokens per thread
  const int per = (a.n_tokens + C::kAllThreads - 1) / C::kAllThreads;
  int64_t mine = 0;
  for (int i = 0; i < per; ++i) {
    const int n = tid * per + i;
    if (n < a.n_tokens) mine += (int64_t)token_of(a, n, C::kKeys).tiles * bundles;
  }
  int64_t inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) warp_sum[warp] = inc;
  if (tid == 0) bits = 0;
  __syncthreads();
  int64_t before = inc - mine, total = 0;
#pragma unroll
  for (int w = 0; w < C::kAllThreads / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  const int64_t ranges = min(total, (int64_t)(a.n_shares >> a.bundle_log2));
  const bool unit_records = by_unit(a);
  if (range >= ranges) {
    if (tid == 0) {
      if (!unit_records) records[share].token = -1;
      words[share] = 0;
    }
    return;
  }
  // The first `longer` ranges have one tile more than the others.
  const int64_t base = (int64_t)((uint64_t)total / (uint32_t)ranges), longer = total - base * ranges;
  const int64_t begin = range * base + min((int64_t)range, longer), end = begin + base + (range < longer);
  if (base >= INT32_MAX) {  // more tiles than a share counts (over 10^13 bytes): refused as a whole
    if (tid == 0) {
      if (!unit_records) records[share].token = -1;
      words[share] = DDTREE_ST_BAD_LENGTH;
    }
    return;
  }
  if (before <= begin && begin < before + mine) {
    int n = tid * per;
    int64_t at = begin - before;
    for (;; ++n) {
      const int64_t here = (int64_t)token_of(a, n, C::kKeys).tiles * bundles;
      if (at < here) break;
      at -= here;
    }
    start_token = n;
    start_at = at;
  }
  __syncthreads();
  const int count = (int)(end - begin);

  // ---- lookups: kStages tiles ahead of the arithmetic, by one warp, two or four keys a lane
  constexpr int kPerLane = C::kKeys / 32;
  int cur = start_token, unit = 0;
  Token tok = token_of(a, cur, C::kKeys);
  const int first_bundle = (int)((uint64_t)start_at / (uint32_t)tok.tiles);
  int tile = (int)(start_at - (int64_t)first_bundle * tok.tiles);
  int kv_head = (first_bundle << a.bundle_log2) + sub;
  bool begun = tile > 0;
  // The token after the current one, loaded when the current one is entered:
  // short contexts change tokens with every tile.
  int next_pos = -1, next_row = 0;
  auto fetch_next = [&] {
    if (cur + 1 < a.n_tokens) {
      next_pos = __ldg(a.positions + cur + 1);
      next_row = row_index(a, cur + 1);
    }
  };
  fetch_next();
  // A tile in two steps, so that the page numbers can be under way meanwhile.
  struct Pages {
    int page[kPerLane];
    int64_t at[kPerLane];  // of the key's row in its page
  };
  auto begin_tile = [&](int i, Pages& p) {
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      const int64_t x = (int64_t)tile * C::kKeys + 32 * k + lane;
      p.page[k] = -1;
      p.at[k] = -1;  // no such key
      if (x < tok.seen) {
        const int j = (int)(x < tok.first ? x : x - tok.first + tok.lo);
        const int number = a.page.quotient(j);
        p.at[k] = (j - number * a.page_size) * a.token_stride + kv_head * a.head_stride;
        p.page[k] = __ldg(a.table + (int64_t)tok.row * a.table_stride + number);
      }
    }
    const bool unit_ends = tile + 1 == tok.tiles, range_ends = i + 1 == count;
    if (lane == 0) {
      Tile t;
      t.token = cur;
      t.kv_head = kv_head;
      t.unit = unit;
      t.flags = (tile == 0 || i == 0 ? kFirst : 0) | (unit_ends || range_ends ? kLast : 0) | (begun ? kBegun : 0) |
                (unit_ends ? 0 : kGoesOn);
      if (C::kTensor && !unit_ends && !range_ends && (tile + 2 == tok.tiles || i + 2 == count)) t.flags |= kNextLast;
      tiles[i % C::kTileRing] = t;
      if (tok.seen == 0) atomicOr(&bits, DDTREE_ST_BAD_LENGTH);
      // The unit's record, where it starts; without units' own, the share's, where the share ends.
      const bool goes_on = range_ends && !unit_ends && !begun;
      if (unit_records ? !begun && (unit_ends || range_ends) : range_ends) {
        Record r;
        r.token = goes_on ? cur : -1;
        r.kv_head = kv_head;
        r.first_share = share;
        const int64_t last = end - 1 + (tok.tiles - 1 - tile);  // the unit's last tile in the list
        const int64_t in_longer = longer * (base + 1);
        r.last_share = (int)(last < in_longer ? last / (base + 1) : longer + (last - in_longer) / base) * (1 << a.bundle_log2) + sub;
        records[unit_records ? cur * a.n_kv_heads + kv_head : share] = r;
      }
    }
    if (unit_ends && !range_ends) {
      tile = 0;
      begun = false;
      ++unit;
      kv_head += 1 << a.bundle_log2;
      if (kv_head >= a.n_kv_heads) {
        kv_head = sub;
        do {
          ++cur;
          tok = token_at(a, next_pos, next_row, C::kKeys);
          fetch_next();
        } while (tok.tiles == 0);
      }
    } else {
      ++tile;
    }
  };
  auto end_tile = [&](int i, const Pages& p) {
    const int slot = i % C::kRing;
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      const bool good = p.page[k] >= 0 && p.page[k] < a.n_pages;
      if (p.at[k] >= 0 && !good) atomicOr(&bits, DDTREE_ST_BAD_INDEX);
      offsets[slot][32 * k + lane] = good ? p.page[k] * a.page_stride + p.at[k] : 0;
      const uint32_t have = __ballot_sync(0xffffffffu, good);
      if (lane == 0) there[slot][k] = have;
    }
  };
  if constexpr (C::kTensor) {
    if (tid < C::kTileRing) tiles[tid] = Tile{start_token, 0, 0, 0};
    if (tid == 0) {
      for (int k = 0; k < C::kStages; ++k) {
        ptx::mbar_init(&tensor.full[k], C::kCopyThreads + 1);
        ptx::mbar_init(&tensor.values[k], 1);
      }
      for (int k = 0; k < 2; ++k) {
        ptx::mbar_init(&tensor.scores[k], 1);
        ptx::mbar_init(&tensor.queries[k], 1);
      }
      ptx::fence_mbar_init();
    }
    if (warp == kAllocWarp) {
      ptx::tmem_alloc(&tensor.base, tmem_cols(kDim));
      ptx::tmem_relinquish();
    }
  }
  if (warp == kWarps) {
    Pages even, odd;
    if constexpr (C::kTensor) {
      // Page numbers are loaded two tiles ahead of the copies: beside those a
      // load takes some 1,000 cycles, about what a tile has (64 rows of 64 columns
      // 206 -> 198 us per GB; four of 131k on pages of one token, 128 columns, 60
      // -> 56; 64 requests of 512 keys 0.5 us slower).
      auto step = [&](int i, Pages& mine, Pages& other) {
        __syncwarp();
        copies_barrier();  // the copies of tile i start; at most kStages + 1 tiles before it are in use
        if (i + 2 < count) begin_tile(i + 2, mine);
        if (i + 1 < count) end_tile(i + 1, other);
      };
      __syncthreads();
      begin_tile(0, even);
      if (count > 1) begin_tile(1, odd);
      end_tile(0, even);
      for (int i = 0; i < count; i += 2) {
        step(i, even, odd);
        if (i + 1 < count) step(i + 1, odd, even);
      }
    } else {
      auto look_up = [&](int i) {
        begin_tile(i, even);
        end_tile(i, even);
      };
      for (int i = 0; i < C::kStages && i < count; ++i) look_up(i);
      __syncthreads();
      for (int i = 0; i < count; ++i) {
        __syncthreads();  // tile i's slot is in use, the one of tile i + kStages free
        if (i + C::kStages < count) look_up(i + C::kStages);
      }
    }
    __syncthreads();
    if (lane == 0) words[share] = bits;
    return;
  }

  // Operands of the tensor core are 64-column slabs of 128-byte rows, swizzled
  // from a 1024-byte border; for ldmatrix a row lies whole.
  const uint32_t p_at = C::kTensor ? (ptx::smem_u32(smem) + 1023) & ~1023u : ptx::smem_u32(smem);
  const uint32_t q_ring = p_at + C::kQAt, ring = p_at + C::kRingAt;
  constexpr int kPitch = C::kTensor ? 128 : C::kRowBytes;
  auto swizzled = [](int row, int chunk, int rows) {
    if constexpr (C::kTensor) return (uint32_t)((chunk >> 3) * rows * 128 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
    else return (uint32_t)(row * C::kRowBytes + ((chunk ^ (row & 7)) << 4));
  };
  // Starts the copies of tile i (kTensor: the barrier follows; else every thread
  // commits a group, empty or not).
  // A thread copies one chunk of every kRowsPerStep-th row: the swizzle of its
  // rows is the same, so shared addresses advance by a constant (steps of four
  // rows: the third bit of the row alternates).
  constexpr int kRowsPerStep = C::kCopyThreads / kChunks;
  static_assert(C::kKeys % kRowsPerStep == 0 && kRowsPerStep % 4 == 0, "copy steps");
  const int copy_tid = C::kTensor ? tid & 127 : tid;
  const int copy_chunk = copy_tid % kChunks, copy_row = copy_tid / kChunks;
  const uint32_t copy_at = swizzled(copy_row, copy_chunk, C::kKeys);
  const uint16_t *copy_k = a.k + 8 * copy_chunk, *copy_v = a.v + 8 * copy_chunk;
  auto start_queries = [&](int i) {
    if (i >= count) return;
    const Tile t = tiles[i % C::kTileRing];
    if (!(t.flags & kFirst)) return;
    const uint32_t q_at = q_ring + (t.unit % C::kQSlots) * C::kQBytes;
    const uint16_t* q = a.q + t.token * a.q_stride + (int64_t)t.kv_head * a.group * kDim;
#pragma unroll
    for (int r = copy_row; r < C::kRows; r += kRowsPerStep)
      ptx::cp_async16_zfill(q_at + swizzled(r, copy_chunk, C::kRows), r < a.group ? q + r * kDim + 8 * copy_chunk : a.q,
                            r < a.group ? 16u : 0u);
  };
  auto start_copies = [&](int i) {
    if (i < count) {
      const int slot = i % C::kRing;
      const uint32_t k_at = ring + (i % C::kStages) * 2 * C::kTileBytes + copy_at, v_at = k_at + C::kTileBytes;
      uint32_t full = 0xffffffffu;
#pragma unroll
      for (int w = 0; w < C::kKeys / 32; ++w) full &= there[slot][w];
      if (full == 0xffffffffu) {
#pragma unroll
        for (int r = 0; r < C::kKeys; r += kRowsPerStep) {
          const int64_t off = offsets[slot][copy_row + r];
          ptx::cp_async16((k_at ^ ((r & 4) << 4)) + r * kPitch, copy_k + off);
          ptx::cp_async16((v_at ^ ((r & 4) << 4)) + r * kPitch, copy_v + off);
        }
      } else {
#pragma unroll 2
        for (int r = 0; r < C::kKeys; r += kRowsPerStep) {
          const int64_t off = offsets[slot][copy_row + r];
          const int key = copy_row + r;
          const uint32_t size = (there[slot][key >> 5] >> (key & 31)) & 1 ? 16u : 0u;
          ptx::cp_async16_zfill((k_at ^ ((r & 4) << 4)) + r * kPitch, copy_k + off, size);
          ptx::cp_async16_zfill((v_at ^ ((r & 4) << 4)) + r * kPitch, copy_v + off, size);
        }
      }
      if constexpr (!C::kTensor) start_queries(i);
    }
    if constexpr (!C::kTensor) asm volatile("cp.async.commit_group;" ::: "memory");
  };

  __syncthreads();
  if constexpr (!C::kTensor) {
#pragma unroll 1
    for (int i = 0; i < C::kStages - 1; ++i) start_copies(i);
  }

  if constexpr (C::kTensor) {
    tensor_tiles<kHalf, kDim, kShort>(a, ws, tensor, p_at, q_ring, ring, tiles, there, &top_s[0][0], reinterpret_cast<float2*>(&sum_s[0][0]), &bits, count, share, start_copies,
                              start_queries);
  } else {
    auto computing_warps = [] { asm volatile("bar.sync 1, %0;" ::"n"(C::kThreads) : "memory"); };

    // ---- this warp's rows (16 of the group) and keys of every tile
    const int wm = warp % kWM, wn = warp / kWM % C::kWN, wk = warp / (kWM * C::kWN);
    constexpr int kWarpKeys = C::kKeys / C::kWK;
    constexpr int kBlock = kWarpKeys < 32 ? 16 : 32;  // keys of one softmax step
    constexpr int kCols = kDim / C::kWN;              // columns of a warp
    // Query fragments in registers for the whole unit, or read again per tile.
    constexpr bool kHoldQ = kDim <= 128;
    uint32_t qf[kHoldQ ? kDim / 16 : 1][4];
    float o[kCols / 8][4], top[2], sum[2];
    // Probabilities meet V in the cache's type: half a step of it each, in exchange
    // for one matrix instruction per product (error of bf16 outputs against 64 bits
    // 0.00164 -> 0.00175, most of it the outputs' own rounding).  The sum takes them
    // unrounded, so the logarithm does not see it.  fp16 holds nothing below 2^-24,
    // so there they carry a factor of 2^10: a key counts down to 2^-34 of the
    // largest, and the factor leaves with the division by the sum.
    constexpr float kShift = kHalf ? 10.f : 0.f;
    // A negative scale turns the products' signs instead; zero becomes the least
    // number, which no product survives, so that absent keys stay at -inf.
    const float scale = fmaxf(fabsf(a.scale_log2), 1.4e-45f);

    // Fragment addresses.  A row's chunks are exchanged by its low three bits,
    // which are the lane's in every matrix it addresses, so four offsets serve
    // all columns and the rest is constant.
    uint32_t k_off[4], v_off[4], q_off[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      k_off[j] = swizzled(wk * kWarpKeys + (lane & 7) + ((lane >> 4) << 3), 2 * j + ((lane >> 3) & 1), C::kKeys);
      v_off[j] = swizzled(wk * kWarpKeys + (lane & 15), 2 * j + (lane >> 4), C::kKeys) + wn * kCols * 2;
      q_off[j] = swizzled(wm * 16 + (lane & 15), 2 * j + (lane >> 4), C::kRows);
    }

    for (int i = 0; i < count; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 2) : "memory");
      __syncthreads();
      start_copies(i + C::kStages - 1);
      const int slot = i % C::kRing;
      const Tile t = tiles[i % C::kTileRing];
      const uint32_t k_at = ring + (i % C::kStages) * 2 * C::kTileBytes, v_at = k_at + C::kTileBytes;
      const uint32_t q_at = q_ring + (t.unit % C::kStages) * C::kQBytes;
      if (t.flags & kFirst) {
        if constexpr (kHoldQ) {
#pragma unroll
          for (int ks = 0; ks < kDim / 16; ++ks) ldsm4(q_at + q_off[ks & 3] + (ks >> 2) * 128, qf[ks]);
        }
#pragma unroll
        for (int d = 0; d < kCols / 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
        top[0] = top[1] = -INFINITY;
        sum[0] = sum[1] = 0.f;
      }
#pragma unroll 1
      for (int block = 0; block < kWarpKeys; block += kBlock) {
        const int key0 = wk * kWarpKeys + block;
        const uint32_t k_blk = k_at + block * C::kRowBytes, v_blk = v_at + block * C::kRowBytes;
        float s[kBlock / 8][4];
#pragma unroll
        for (int x = 0; x < kBlock / 8; ++x) s[x][0] = s[x][1] = s[x][2] = s[x][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < kDim / 16; ++ks) {
          uint32_t again[4];
          if constexpr (!kHoldQ) ldsm4(q_at + q_off[ks & 3] + (ks >> 2) * 128, again);
          const uint32_t(&af)[4] = kHoldQ ? qf[kHoldQ ? ks : 0] : again;
#pragma unroll
          for (int x = 0; x < kBlock / 16; ++x) {
            uint32_t b[4];
            ldsm4(k_blk + k_off[ks & 3] + (ks >> 2) * 128 + x * 16 * C::kRowBytes, b);
            mma<kHalf>(s[2 * x], af, b[0], b[1]);
            mma<kHalf>(s[2 * x + 1], af, b[2], b[3]);
          }
        }
        // Products as they are, keys that are not there at -inf; the scale (made
        // positive, see below) enters with the maximum in one multiply-add.
        const uint32_t mask = there[slot][key0 >> 5] >> (key0 & 31);
        constexpr uint32_t kAll = kBlock == 32 ? 0xffffffffu : (1u << (kBlock & 31)) - 1;
        float high[2] = {top[0], top[1]};
        if (a.scale_log2 < 0.f) {
#pragma unroll
          for (int x = 0; x < kBlock / 8; ++x) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[x][e] = -s[x][e];
          }
        }
        if ((mask & kAll) != kAll) {
#pragma unroll
          for (int x = 0; x < kBlock / 8; ++x) {
            const uint32_t two = mask >> (8 * x + 2 * (lane & 3));
            if (!(two & 1)) s[x][0] = s[x][2] = -INFINITY;
            if (!(two & 2)) s[x][1] = s[x][3] = -INFINITY;
          }
        }
#pragma unroll
        for (int x = 0; x < kBlock / 8; ++x) {
          high[0] = fmaxf(high[0], fmaxf(s[x][0], s[x][1]));
          high[1] = fmaxf(high[1], fmaxf(s[x][2], s[x][3]));
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          high[r] = fmaxf(high[r], __shfl_xor_sync(0xffffffffu, high[r], 1));
          high[r] = fmaxf(high[r], __shfl_xor_sync(0xffffffffu, high[r], 2));
        }
        if (__any_sync(0xffffffffu, high[0] > top[0] || high[1] > top[1])) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float keep = top[r] == -INFINITY ? 0.f : power2((top[r] - high[r]) * scale);
            sum[r] *= keep;
            top[r] = high[r];
#pragma unroll
            for (int d = 0; d < kCols / 8; ++d) {
              o[d][2 * r] *= keep;
              o[d][2 * r + 1] *= keep;
            }
          }
        }
        const float base[2] = {top[0] == -INFINITY ? 0.f : kShift - top[0] * scale, top[1] == -INFINITY ? 0.f : kShift - top[1] * scale};
#pragma unroll
        for (int x = 0; x < kBlock / 8; ++x) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[x][e] = power2(fmaf(s[x][e], scale, base[e >> 1]));
          sum[0] += s[x][0] + s[x][1];
          sum[1] += s[x][2] + s[x][3];
        }
#pragma unroll
        for (int x = 0; x < kBlock / 16; ++x) {
          const uint32_t p[4] = {pack2<kHalf>(s[2 * x][0], s[2 * x][1]), pack2<kHalf>(s[2 * x][2], s[2 * x][3]),
                                 pack2<kHalf>(s[2 * x + 1][0], s[2 * x + 1][1]), pack2<kHalf>(s[2 * x + 1][2], s[2 * x + 1][3])};
#pragma unroll
          for (int d = 0; d < kCols / 16; ++d) {
            uint32_t b[4];
            ldsm4_trans(v_blk + v_off[d & 3] + (d >> 2) * 128 + x * 16 * C::kRowBytes, b);
            mma<kHalf>(o[2 * d], p, b[0], b[1]);
            mma<kHalf>(o[2 * d + 1], p, b[2], b[3]);
          }
        }
      }
      if (!(t.flags & kLast)) continue;

      // ---- the unit ends here: join the warps' rows through this tile's stage
      computing_warps();  // every warp is done with the tile
      float* rows = reinterpret_cast<float*>(smem + (i % C::kStages) * 2 * C::kTileBytes);
      // Row r of key part w; the exchange of column groups keeps the four rows that lanes write at once on other banks.
      auto cell = [&](int w, int r, int col) { return rows + (w * C::kRows + r) * kDim + (col ^ ((r & 3) << 3)); };
      const int g = lane >> 2;
      const bool whole = !(t.flags & (kBegun | kGoesOn));
      const int64_t part = 2 * share + (t.flags & kBegun ? 0 : 1);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
        const int row = wm * 16 + g + 8 * r;
        if ((lane & 3) == 0 && wn == 0) {
          top_s[wk][row] = top[r] == -INFINITY ? top[r] : top[r] * scale;  // from here on in base 2
          sum_s[wk][row] = sum[r];
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = wm * 16 + g + 8 * r;
        if (row >= a.group) continue;
#pragma unroll
        for (int d = 0; d < kCols / 8; ++d) {
          const int col = wn * kCols + 8 * d;
          *reinterpret_cast<float2*>(cell(wk, row, col + 2 * (lane & 3))) = make_float2(o[d][2 * r], o[d][2 * r + 1]);
        }
      }
      computing_warps();
      // Columns of a thread: few where many threads share a small group's rows
      // (185k single 69.3 -> 67.1 us with four of 256; with 128 threads four
      // spill where eight do not: 1024 requests of 100 keys 109 us instead of 92).
      constexpr int kVec = kThreads == 128 ? 8 : 4;
      for (int e = tid; e < a.group * (kDim / kVec); e += kThreads) {
        const int row = e / (kDim / kVec), col = (e - row * (kDim / kVec)) * kVec;
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int k = 0; k < C::kWK; ++k) m = fmaxf(m, top_s[k][row]);
        const float from = m == -INFINITY ? 0.f : m;
        float4 x[kVec / 4];
#pragma unroll
        for (int q = 0; q < kVec / 4; ++q) x[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < C::kWK; ++k) {
          const float w = power2(top_s[k][row] - from);
          l += w * sum_s[k][row];
#pragma unroll
          for (int q = 0; q < kVec / 4; ++q) {
            const float4 u = *reinterpret_cast<const float4*>(cell(k, row, col + 4 * q));
            x[q].x += w * u.x; x[q].y += w * u.y; x[q].z += w * u.z; x[q].w += w * u.w;
          }
        }
        if (whole) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          const int head = t.kv_head * a.group + row;
          uint32_t packed[kVec / 2];
#pragma unroll
          for (int q = 0; q < kVec / 4; ++q) {
            packed[2 * q] = pack2<kHalf>(x[q].x * inv, x[q].y * inv);
            packed[2 * q + 1] = pack2<kHalf>(x[q].z * inv, x[q].w * inv);
          }
          uint16_t* to = a.out + t.token * a.out_stride + (int64_t)head * kDim + col;
          if constexpr (kVec == 8) *reinterpret_cast<uint4*>(to) = make_uint4(packed[0], packed[1], packed[kVec / 2 - 2], packed[kVec / 2 - 1]);
          else *reinterpret_cast<uint2*>(to) = make_uint2(packed[0], packed[1]);
          if (a.lse && col == 0)
            a.lse[(int64_t)t.token * a.n_heads + head] = l == 0.f ? -INFINITY : (m - kShift + log2f(l)) * 0.6931471805599453f;
        } else {
          float4* to = reinterpret_cast<float4*>(a.ws + ws.rows) + (part * C::kRows + row) * (kDim / 4) + col / 4;
#pragma unroll
          for (int q = 0; q < kVec / 4; ++q) to[q] = x[q];
          if (col == 0) reinterpret_cast<float2*>(a.ws + ws.sums)[part * C::kRows + row] = make_float2(m, l);
        }
      }
      // The next iteration's barrier comes before this stage is filled again.
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  if constexpr (C::kTensor) {
    ptx::tc_fence_after();
    if (warp == kAllocWarp) ptx::tmem_dealloc(tensor.base, tmem_cols(kDim));
  }
}

// Joins the parts of the units that go on across shares: a CTA per record (x)
// and slice of the group's rows (y); one more x gathers the status words.
// Eight teams of kDim / 4 threads, a float4 each: they take rows of their own,
// or several share a row's parts; every team keeps its own running maximum, so
// sums and rows are loaded together.
template <bool kHalf, int kDim>
__global__ void __launch_bounds__(2 * kDim) draft_join_kernel(const __grid_constant__ DraftAttnArgs a, int slice_rows) {
  constexpr int kTeams = 8, kLanes = kDim / 4, kUnroll = 8;
  constexpr int kThreads = kTeams * kLanes;
  __shared__ float4 acc[kTeams][kLanes];
  __shared__ float2 team_sum[kTeams];
  const int tid = threadIdx.x;
  const Layout ws = layout_of(a.row_tile, kDim, a.n_shares);
  const int x = blockIdx.x, slice = blockIdx.y;
  const int records = by_unit(a) ? a.n_tokens * a.n_kv_heads : a.n_shares;
  await_grid();
  if (x == records) {
    if (slice > 0) return;
    uint32_t b = 0;
    for (int s = tid; s < a.n_shares; s += kThreads) b |= reinterpret_cast<const uint32_t*>(a.ws + ws.words)[s];
    __shared__ uint32_t all;
    if (tid == 0) all = 0;
    __syncthreads();
    if (b) atomicOr(&all, b);
    __syncthreads();
    if (tid == 0) *reinterpret_cast<uint32_t*>(a.ws) = all;
    return;
  }
  // A padding token's units are in no share and nobody wrote their records; what
  // lies there is loaded (with the position, not after it) and dropped.  Bounds
  // hold for every record that was written; a refused call writes none.
  const Record r = reinterpret_cast<const Record*>(a.ws + ws.records)[x];
  const bool padding = by_unit(a) && __ldg(a.positions + x / a.n_kv_heads) == -1;
  if (padding || r.token < 0 || r.token >= a.n_tokens || r.kv_head < 0 || r.kv_head >= a.n_kv_heads || r.first_share < 0 ||
      r.last_share < r.first_share || r.last_share >= a.n_shares)
    return;
  const int first = r.first_share, parts = ((r.last_share - first) >> a.bundle_log2) + 1;
  const float2* sums = reinterpret_cast<const float2*>(a.ws + ws.sums);
  const float4* rows = reinterpret_cast<const float4*>(a.ws + ws.rows);
  // Part p of the unit, in every bundle-th share: the second place of the first one, the first place of the others.
  auto place = [&](int p, int row) { return ((int64_t)2 * (first + (p << a.bundle_log2)) + (p == 0)) * a.row_tile + row; };
  const int team = tid / kLanes, c = tid - team * kLanes;
  const int row_begin = slice * slice_rows, row_end = min(row_begin + slice_rows, a.group);
  // Teams of a row: as many as the CTA's rows leave, where a row has more parts
  // than one team loads at once.
  const int per_row = parts <= kUnroll || slice_rows > 4 ? 1 : slice_rows > 2 ? 2 : slice_rows > 1 ? 4 : 8;
  for (int row0 = row_begin; row0 < row_end; row0 += kTeams / per_row) {
    const int row = row0 + team / per_row;
    float high = -INFINITY, total = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = team % per_row; p0 < parts && row < row_end; p0 += per_row * kUnroll) {
      float2 s[kUnroll];
      float4 v[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int p = p0 + u * per_row;
        s[u] = make_float2(-INFINITY, 0.f);
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p < parts) {
          s[u] = sums[place(p, row)];
          v[u] = rows[place(p, row) * kLanes + c];
        }
      }
      float top = high;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) top = fmaxf(top, s[u].x);
      const float from = top == -INFINITY ? 0.f : top, keep = power2(high - from);
      total *= keep;
      o.x *= keep; o.y *= keep; o.z *= keep; o.w *= keep;
      high = top;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const float w = power2(s[u].x - from);
        total += w * s[u].y;
        o.x += w * v[u].x; o.y += w * v[u].y; o.z += w * v[u].z; o.w += w * v[u].w;
      }
    }
    if (per_row > 1) {  // the same in the whole CTA
      acc[team][c] = o;
      if (c == 0) team_sum[team] = make_float2(high, total);
      __syncthreads();
      if (team % per_row == 0) {
        for (int k = 0; k < per_row; ++k) high = fmaxf(high, team_sum[team + k].x);
        const float from = high == -INFINITY ? 0.f : high;
        o = make_float4(0.f, 0.f, 0.f, 0.f);
        total = 0.f;
        for (int k = 0; k < per_row; ++k) {
          const float w = power2(team_sum[team + k].x - from);
          const float4 v = acc[team + k][c];
          total += w * team_sum[team + k].y;
          o.x += w * v.x; o.y += w * v.y; o.z += w * v.z; o.w += w * v.w;
        }
      }
      __syncthreads();
    }
    if (team % per_row == 0 && row < row_end) {
      const float inv = total == 0.f ? 0.f : 1.f / total;
      const int head = r.kv_head * a.group + row;
      *reinterpret_cast<uint2*>(a.out + r.token * a.out_stride + (int64_t)head * kDim + 4 * c) =
          make_uint2(pack2<kHalf>(o.x * inv, o.y * inv), pack2<kHalf>(o.z * inv, o.w * inv));
      constexpr float kShift = kHalf ? 10.f : 0.f;
      if (a.lse && c == 0)
        a.lse[(int64_t)r.token * a.n_heads + head] = total == 0.f ? -INFINITY : (high - kShift + log2f(total)) * 0.6931471805599453f;
    }
  }
}

template <bool kHalf, int kDim, int kWM, bool kShort = false>
cudaError_t launch(const DraftAttnArgs& a, cudaStream_t stream) {
  using C = Config<kDim, kWM>;
  // The shared-memory limit belongs to the kernel on a device: set once on each.
  static std::atomic<uint64_t> have{0};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (device & 63);
  if (!(have.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(draft_attn_kernel<kHalf, kDim, kWM, kShort>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    have.fetch_or(bit, std::memory_order_release);
  }
  e = launch_early(draft_attn_kernel<kHalf, kDim, kWM, kShort>, a.n_shares, C::kAllThreads, C::kSmem, stream, a);
  if (e != cudaSuccess) return e;
  // Rows get CTAs of their own where records are few, for their units have many
  // parts (one CTA for all rows: window 12.0 us instead of 8.0, 185k single 85.6
  // instead of 69.7); many records have few parts each, and one CTA takes all
  // rows (64 requests of 512 keys: 31.8 us, with four times the CTAs 35.9).
  const int records = by_unit(a) ? a.n_tokens * a.n_kv_heads : a.n_shares;
  const int slices = std::max(1, std::min(a.group, a.n_shares / records));
  const int slice_rows = (a.group + slices - 1) / slices;
  return launch_early(draft_join_kernel<kHalf, kDim>, dim3(records + 1, (a.group + slice_rows - 1) / slice_rows), 2 * kDim, 0,
                      stream, a, slice_rows);
}

template <bool kHalf, int kDim>
cudaError_t launch_rows(const DraftAttnArgs& a, cudaStream_t stream) {
  if (a.row_tile == 16) return launch<kHalf, kDim, 1>(a, stream);
  if constexpr (kDim == 64) {
    if (a.row_tile == 32) return launch<kHalf, kDim, 2>(a, stream);
  }
  return a.wait_ns < kShortNs ? launch<kHalf, kDim, 4, true>(a, stream) : launch<kHalf, kDim, 4>(a, stream);
}

template <bool kHalf>
cudaError_t launch_dim(const DraftAttnArgs& a, cudaStream_t stream) {
  return a.head_dim == 64    ? launch_rows<kHalf, 64>(a, stream)
         : a.head_dim == 128 ? launch_rows<kHalf, 128>(a, stream)
                             : launch_rows<kHalf, 256>(a, stream);
}

}  // namespace

int draft_row_tile(int group, int head_dim) { return group <= 16 ? 16 : group <= 32 && head_dim == 64 ? 32 : 64; }

int draft_tile_keys(int row_tile, int head_dim) { return keys_of(row_tile, head_dim); }

int draft_shares(int row_tile, int head_dim, int num_sms) { return ctas_of(row_tile, head_dim) * num_sms; }

int64_t draft_workspace_bytes(int row_tile, int head_dim, int n_shares) {
  return (layout_of(row_tile, head_dim, n_shares).total + 255) / 256 * 256;
}

cudaError_t launch_draft_attention(const DraftAttnArgs& a, cudaStream_t stream) {
  return a.dtype == DDTREE_FP16 ? launch_dim<true>(a, stream) : launch_dim<false>(a, stream);
}

}  // namespace ddtree
