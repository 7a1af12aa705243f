// The drafter's attention of one new token per request over its cache in 8 bits
// (include/ddtree_draft8.h).
//
//   s_j = scale ks_j <q, kc_j>,  out = sum_j e^(s_j - m) vs_j vc_j / sum_j e^(s_j - m)
//
// with codes kc, vc and their blocks' scales ks, vs.  As with 16 bits the work
// is a stream of keys, and HBM the bound; half the bytes a key leave an SM half
// the time for its arithmetic.  What carries it:
//
//  - The list of tiles, the equal shares and the join of units that cross shares
//    are those of the 16-bit kernel (k_draft_attn.cu).  Groups of more than 16
//    query heads are several units of 16, side by side in the list, which read the
//    same keys at the same time.
//  - Every warp has 32 keys of a tile to itself, from the page numbers and the
//    copies to the sums, and waits for no other before the unit ends: a lookup warp
//    and barriers for each tile, as with 16 bits, took 209 us for eight requests of
//    1k to 185k (8 x 128 columns) where this takes 117.  Where a row has 256
//    columns two warps share 32 keys, a half of the columns each, since one would
//    hold 128 registers of results.
//  - e4m3 numbers are exact in fp16, so a pair is converted by one instruction
//    and meets fp16 matrix instructions.  A query row moves by a power of two
//    into fp16's range, exactly but for what is 2^-39 of its largest element.
//  - Which column is which in a product's inner dimension is free, as long as
//    both sides agree: a lane takes 16 columns of a key in one load and uses
//    four of them per instruction.  Of V it takes 16 columns (8 where there are
//    64) of the four keys that its probabilities belong to, and pairs of keys are
//    put together by byte permutes; the lane's columns of the result lie next to
//    each other.
//  - Scales stay out of the products.  ks_j multiplies a score; vs_j goes into
//    the exponent: with x_j = s_j + log2 vs_j (in base 2), M = max x_j,
//    O = sum 2^(x_j - M) vc_j,  l = sum 2^(x_j - M) / vs_j,  out = O / l.
//    So what is rounded to fp16 is a row's weight in the result, whatever the
//    scales are.  A key that is not there has ks = 0, log2 vs = -inf and
//    1 / vs = 0, and needs no mask.
//  - What costs now is instructions: two for a pair of codes (K 1.5), and per key
//    its lookup, scales and softmax, some 550 a warp and 32 keys of 64 columns.
//    Pairs of scores go through two-number instructions, and O is scaled only when
//    a maximum has grown well.
//
// Measured (calls back to back; the share is of the copy rate of 6.7 TB/s): the
// eight requests above (738 MB) 117 us, 0.94; 61 requests of 0.5k to 16k, 8 x 64
// columns of fp16 (292 MB) 64 to 66 us, 0.67: the issue slots of an SM are 60 % busy
// and the conversions' pipe is the next, and rows 8 to 15 of a product, empty here,
// are computed as well; one of 185k with 2 x 256 columns (194 MB) 46, 0.63: some 8 us
// of it the lists, the joins and the launches; a window of 2,048 at 65k 9.1, where the
// 16-bit kernel takes 8.3: steps that wait for each other, in two grids, and no bytes
// to save.  Every 16 query heads of a key head convert its codes again: eight requests
// of 65,536, 32,768 and 16,384 keys (8 x 64, 8 x 128 and 4 x 256 columns) take 106, 96
// and 62 us with 16 heads a key head (16 bits 161, 158, 89), 199, 154 and 91 with 32
// (181, 168, 97) and 385, 293 and 165 with 64 (195, 172, 100, on tensor memory).
#include <atomic>

#include "f32x2.cuh"
#include "rope.cuh"
#include "tc_ptx.cuh"

namespace ddtree {
namespace {

constexpr int kWarps = 4;       // of a CTA, each with keys of its own
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 16;       // query heads of a unit
// A weight carries a factor of 2^kShift in fp16, and the maximum that it is
// relative to moves only when it has grown by more than 2^kGrowth: 2^15 is the
// largest weight, and one counts down to 2^-34 of it.
constexpr float kShift = 10.f, kGrowth = 5.f;
// Products cut their sums off where they do not fit into 32 bits, always towards zero:
// 4e-9 of it for every key of a warp (values of one sign), which with a million keys in
// one share was 0.1 % (0.23 % with 256 columns).  So after this many tiles, 8,192 keys of
// a warp, the sums start anew, and what they were is added up in the workspace.  Where
// no unit has more tiles, another form leaves that out (61 requests of 0.5k to 16k, 8 x
// 64 columns: 64.5 us for 66.1 in turn).
constexpr int kChain = 256;

template <int kDim>
struct Config {
  // 256 columns are halved between two warps, which add up their halves of the scores.
  static constexpr int kHalves = kDim == 256 ? 2 : 1, kCols = kDim / kHalves;
  static constexpr int kWarpKeys = 32;                      // of a tile, for each warp or pair
  static constexpr int kParts = kWarps / kHalves, kKeys = kParts * kWarpKeys;
  static constexpr int kCtas = kDim == 64 ? 4 : 3;          // per SM
  static constexpr int kStages = kDim == 64 ? 3 : 2;
  static constexpr int kHalfBytes = kWarpKeys * kCols;      // a warp's K of a tile, and its V
  static constexpr int kStageBytes = 2 * kHalfBytes;
  static constexpr int kSmem = kWarps * kStages * kStageBytes;
  static_assert(kStageBytes == kRows * kCols * 4, "a warp's rows are joined in the stage just consumed");
};

// A unit that goes on from one share to others: where its parts lie (a record
// per unit where units are no more than shares, else one per share, for the unit
// that starts there and goes on; token -1: nothing to join).
struct Record {
  int32_t token, head, first_share, last_share;
};
__host__ __device__ inline bool by_unit(const Draft8AttnArgs& a) { return (int64_t)a.n_tokens * a.unit_heads <= a.n_shares; }

// Workspace: status block, per share a status word and a record, then the
// (maximum, sum) pairs and the rows of two partial units per share; and of what a
// share holds of a long unit (pairs twice, taken in turn).
struct Layout {
  int64_t words, records, sums, rows, held_sums, held_rows, total;
};
__host__ __device__ inline Layout layout_of(int dim, int shares) {
  Layout l;
  l.words = 256;
  l.records = l.words + ((int64_t)shares * 4 + 255) / 256 * 256;
  l.sums = l.records + ((int64_t)shares * 16 + 255) / 256 * 256;
  l.rows = l.sums + ((int64_t)shares * 2 * kRows * 8 + 255) / 256 * 256;
  l.held_sums = l.rows + (int64_t)shares * 2 * kRows * dim * 4;
  l.held_rows = l.held_sums + (int64_t)shares * 2 * kRows * 8;
  l.total = l.held_rows + (int64_t)shares * kRows * dim * 4;
  return l;
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four codes as fp16 pairs.
__device__ __forceinline__ void from_codes(uint32_t c, uint32_t& lo, uint32_t& hi) {
  asm("{ .reg .b16 a, b;\n"
      "  mov.b32 {a, b}, %2;\n"
      "  cvt.rn.f16x2.e4m3x2 %0, a;\n"
      "  cvt.rn.f16x2.e4m3x2 %1, b; }"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float power2(float x) { return ptx::ex2_approx(x); }
// Byte offset of a 16-byte chunk of a key in its tile.  128-byte lines keep
// their chunks exchanged so that the eight lanes of a load's quarter meet eight
// different ones: for K, lanes with four chunks of two neighbouring keys; for V,
// lanes with two chunks of every second of eight keys.
template <int kDim>
__device__ __forceinline__ uint32_t k_at(int key, int chunk) {
  if constexpr (kDim == 64) return (uint32_t)(key * 64 + chunk * 16);
  else return (uint32_t)(key * kDim + ((chunk ^ ((key & 1) << 2)) << 4));
}
template <int kDim>
__device__ __forceinline__ uint32_t v_at(int key, int chunk) {
  if constexpr (kDim == 64) return (uint32_t)((key >> 1) * 128 + (((((key & 1) << 2) + chunk) ^ (((key >> 1) & 3) << 1)) << 4));
  else return (uint32_t)(key * kDim + ((chunk ^ (((key >> 1) & 3) << 1)) << 4));
}

// What a token sees, from its position and table row.
struct Token {
  int pos, row, lo, first, tiles;  // window start, sinks before it, tiles per unit (0: padding)
  int64_t seen;                    // visible keys (0 of a token whose data is bad: one empty tile)
};
__device__ __forceinline__ int row_index(const Draft8AttnArgs& a, int n) { return a.token_rows ? __ldg(a.token_rows + n) : n; }
__device__ __forceinline__ Token token_at(const Draft8AttnArgs& a, int pos, int row, int tile_keys) {
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
__device__ __forceinline__ Token token_of(const Draft8AttnArgs& a, int n, int tile_keys) {
  return token_at(a, __ldg(a.positions + n), row_index(a, n), tile_keys);
}

// Query heads of a unit: the first one, and how many.
__device__ __forceinline__ int first_head(const Draft8AttnArgs& a, int head, int& rows) {
  const int kv = head / a.row_tiles, part = head - kv * a.row_tiles;
  rows = min(kRows, a.group - part * kRows);
  return kv * a.group + part * kRows;
}

template <bool kHalf, int kDim, bool kLong>
__global__ void __launch_bounds__(kThreads, Config<kDim>::kCtas) draft8_attn_kernel(const __grid_constant__ Draft8AttnArgs a) {
  using C = Config<kDim>;
  constexpr int kStages = C::kStages, kWarpKeys = C::kWarpKeys, kCols = C::kCols;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t offsets[kWarps][32];                  // byte offset of a key's row
  // Of a tile's keys: scale of K, log2 of that of V, its inverse.
  __shared__ __align__(16) float k_scales[kWarps][32], v_log2[kWarps][32], v_inverse[kWarps][32];
  __shared__ float top_s[C::kParts][kRows], sum_s[C::kParts][kRows];
  __shared__ int64_t warp_sum[kWarps];
  __shared__ int start_token;
  __shared__ int64_t start_at;
  __shared__ uint32_t bits;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int share = blockIdx.x, range = share >> a.bundle_log2, sub = share - (range << a.bundle_log2);
  const int bundles = a.unit_heads >> a.bundle_log2;
  const Layout ws = layout_of(kDim, a.n_shares);
  Record* records = reinterpret_cast<Record*>(a.ws + ws.records);
  uint32_t* words = reinterpret_cast<uint32_t*>(a.ws + ws.words);
  release_grid();
  await_grid();

  // ---- the list of tiles: sums over the tokens, a run of tokens per thread
  const int per = (a.n_tokens + kThreads - 1) / kThreads;
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
  for (int w = 0; w < kWarps; ++w) {
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

  // ---- the walk along the list, by every warp for itself: a tile is found some
  // turns before it is computed, first its keys' page numbers, then, when they are
  // here, its rows' offsets, the copies and the loads of the scales
  struct Spot {                       // the next tile to be found
    int token, head, tile;
    Token tok;
    const int32_t* pages;
    uint32_t seen;
    int behind;                       // keys between the sinks and the window
  } at;
  auto enter = [&](const Token& t) {
    at.tok = t;
    at.pages = a.table + (uint64_t)(uint32_t)t.row * (uint32_t)a.table_stride;
    at.seen = (uint32_t)t.seen;
    at.behind = t.lo - t.first;
  };
  at.token = start_token;
  enter(token_of(a, at.token, C::kKeys));
  {
    const int first_bundle = (int)((uint64_t)start_at / (uint32_t)at.tok.tiles);
    at.tile = (int)(start_at - (int64_t)first_bundle * at.tok.tiles);
    at.head = (first_bundle << a.bundle_log2) + sub;
  }
  int next_pos = -1, next_row = 0;    // of the token behind it, loaded when it is entered
  auto fetch_next = [&] {
    if (at.token + 1 < a.n_tokens) {
      next_pos = __ldg(a.positions + at.token + 1);
      next_row = row_index(a, at.token + 1);
    }
  };
  fetch_next();
  const int part = warp / C::kHalves, half = warp % C::kHalves;  // keys and columns of this warp
  const int key_lane = part * kWarpKeys + lane;                    // this lane's key of a tile
  int page = -1, place = -1, kv_head = 0;  // of the tile found last; place -1: no such key
  uint64_t head_at = 0;                    // its key head's place in a token, in 16 bytes
  auto find = [&] {
    kv_head = a.row_tiles == 1 ? at.head : at.head / a.row_tiles;
    head_at = (uint64_t)(uint32_t)kv_head * a.head_step;
    const uint32_t x = (uint32_t)at.tile * C::kKeys + key_lane;  // below 2^31 + kKeys
    place = -1;
    page = -1;
    if (x < at.seen) {
      const int j = (int)x + ((int)x < at.tok.first ? 0 : at.behind);
      const int number = a.page.quotient(j);
      place = j - number * a.page_size;
      page = __ldg(at.pages + number);
    }
    if (at.tok.seen == 0 && tid == 0) atomicOr(&bits, DDTREE_ST_BAD_LENGTH);
    if (++at.tile == at.tok.tiles) {
      at.tile = 0;
      at.head += 1 << a.bundle_log2;
      if (at.head >= a.unit_heads) {
        at.head = sub;
        do {
          if (++at.token >= a.n_tokens) break;  // behind the list's end nothing is found any more
          enter(token_at(a, next_pos, next_row, C::kKeys));
          fetch_next();
        } while (at.tok.tiles == 0);
      }
    }
  };
  const uint32_t ring = ptx::smem_u32(smem) + warp * kStages * C::kStageBytes;
  constexpr int kChunks = kCols / 16, kRowsPerStep = 32 / kChunks;
  const int copy_chunk = lane % kChunks, copy_row = lane / kChunks;
  const uint8_t *k_src = a.k + half * kCols + 16 * copy_chunk, *v_src = a.v + half * kCols + 16 * copy_chunk;
  const uint32_t copy_k = ring + k_at<kCols>(copy_row, copy_chunk), copy_v = ring + C::kHalfBytes + v_at<kCols>(copy_row, copy_chunk);
  // Scales of the tiles under way (0: no key), newest last.
  float ks[kStages], vs[kStages];
  bool has[kStages];
  auto start = [&](int slot) {  // the copies of the tile found last
    const bool good = page >= 0 && page < a.n_pages;
    if (place >= 0 && !good) atomicOr(&bits, DDTREE_ST_BAD_INDEX);
    ks[kStages - 1] = vs[kStages - 1] = 0.f;
    has[kStages - 1] = good;
    int64_t off = -1;
    if (good) {
      off = ((uint64_t)(uint32_t)page * a.page_step + (uint64_t)(uint32_t)place * a.token_step + head_at) << 4;
      const uint32_t block = (uint32_t)page * a.blocks + a.block.quotient(place);  // below n_pages * page_size
      const uint64_t s = (uint64_t)block * (uint32_t)a.n_kv_heads + kv_head;
      ks[kStages - 1] = a.k_scale[s];
      vs[kStages - 1] = a.v_scale[s];
    }
    __syncwarp();  // the offsets of the last tile are used, and its stage
    offsets[warp][lane] = off;
    const bool full = __all_sync(0xffffffffu, good);
    __syncwarp();
    // Steps of four rows turn one bit of the exchange of chunks of V, steps of eight leave it as it is.
    const uint32_t k_to = copy_k + slot * C::kStageBytes, v_to = copy_v + slot * C::kStageBytes;
    constexpr int kSteps = kWarpKeys / kRowsPerStep;
    int64_t o[kSteps];
#pragma unroll
    for (int r = 0; r < kSteps; ++r) o[r] = offsets[warp][r * kRowsPerStep + copy_row];
    if (full) {
#pragma unroll
      for (int r = 0; r < kSteps; ++r) {
        const uint32_t turned = kCols > 64 ? (r * kRowsPerStep & 4) << 4 : 0;
        ptx::cp_async16(k_to + r * kRowsPerStep * kCols, k_src + o[r]);
        ptx::cp_async16((v_to ^ turned) + r * kRowsPerStep * kCols, v_src + o[r]);
      }
    } else {
#pragma unroll
      for (int r = 0; r < kSteps; ++r) {
        const uint32_t turned = kCols > 64 ? (r * kRowsPerStep & 4) << 4 : 0, size = o[r] < 0 ? 0u : 16u;
        ptx::cp_async16_zfill(k_to + r * kRowsPerStep * kCols, k_src + (o[r] < 0 ? 0 : o[r]), size);
        ptx::cp_async16_zfill((v_to ^ turned) + r * kRowsPerStep * kCols, v_src + (o[r] < 0 ? 0 : o[r]), size);
      }
    }
  };
  auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
  auto pair_of_warps = [&] { asm volatile("bar.sync %0, 64;" ::"r"(2 + part) : "memory"); };
  auto all_warps = [] { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); };

  // The tile that is computed, apart from the one that is found.
  int token = at.token, head = at.head, tile = at.tile;
  Token now = at.tok;
  bool begun = tile > 0;
  // Each turn's copies need the page numbers found a turn before.
  find();
#pragma unroll
  for (int i = 0; i < kStages; ++i) {
#pragma unroll
    for (int k = 0; k + 1 < kStages; ++k) {
      ks[k] = ks[k + 1];
      vs[k] = vs[k + 1];
      has[k] = has[k + 1];
    }
    if (i < count) start(i);
    commit();
    if (i + 1 < count) find();
  }

  // ---- this warp's keys of every tile
  const int g = lane >> 2, q4 = lane & 3;
  constexpr int kGroups = kWarpKeys / 8;     // of eight keys
  constexpr int kChunkCols = kCols / 8;      // columns of V that a lane reads at once
  constexpr int kTilesN = kCols / 8;         // product tiles of eight columns
  uint32_t qf[kCols / 16][4];
  // Where this lane's codes lie in a stage; chunks of the other half of 128 bytes are 64 away, either way.
  const uint32_t k_lane = ring + k_at<kCols>(g, q4);
  const uint32_t v_lane = ring + C::kHalfBytes + (kCols == 64 ? v_at<kCols>(2 * q4, g >> 1) + (g & 1) * 8 : v_at<kCols>(2 * q4, g));
  float o[kTilesN][4], top[2], factor[2];
  uint64_t sum[2];
  bool first = true;
  int rows = 0, head0 = 0, chain = 0, held = 0;  // tiles in the sums, times that the unit's sums have gone to the workspace

  for (int i = 0; i < count; ++i) {
    const int slot = i % kStages;
    const bool unit_ends = tile + 1 == now.tiles, last = unit_ends || i + 1 == count;
    const bool joins = last || (kLong && ++chain == kChain);
    if (first) {
      // Queries: columns 16 q4 .. 16 q4 + 15 of every 64, of rows g and g + 8, four of them an instruction.
      head0 = first_head(a, head, rows);
      const uint16_t* q = a.q + token * a.q_stride + (int64_t)head0 * kDim;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint4* src = reinterpret_cast<const uint4*>(q + (int64_t)(g + 8 * r) * kDim) + 2 * q4;
        const bool live = g + 8 * r < rows;
        uint4 v[kDim / 32];
        float most = 0.f;
#pragma unroll
        for (int b = 0; b < kDim / 32; ++b) v[b] = live ? src[(b >> 1) * 8 + (b & 1)] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int b = 0; b < kDim / 32; ++b) {
          float x[8];
          unpack8<kHalf>(v[b], x);
#pragma unroll
          for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(x[e]));
        }
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        // The largest element to [2^14, 2^15); of bf16 they reach 2^128.
        const int up = most == 0.f ? 0 : max(-114, min(120, 14 + 127 - (int)(__float_as_uint(most) >> 23)));
        const float by = __uint_as_float((uint32_t)(up + 127) << 23);
        factor[r] = __uint_as_float((uint32_t)(127 - up) << 23) * a.scale_log2;
#pragma unroll
        for (int b = 0; b < kCols / 32; ++b) {
          float x[8];
          if constexpr (C::kHalves == 2) unpack8<kHalf>(half ? v[b + kCols / 32] : v[b], x);
          else unpack8<kHalf>(v[b], x);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            qf[2 * b + e][r] = pack2<true>(x[4 * e] * by, x[4 * e + 1] * by);
            qf[2 * b + e][2 + r] = pack2<true>(x[4 * e + 2] * by, x[4 * e + 3] * by);
          }
        }
      }
#pragma unroll
      for (int d = 0; d < kTilesN; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
      top[0] = top[1] = -INFINITY;
      sum[0] = sum[1] = 0;
    }
    // Scales, a key a lane; they came with the copies before the last ones.
    uint32_t out;
    __syncwarp();  // those of the last tile are used
    {
      const bool good = ks[0] >= 0x1p-64f && ks[0] <= 0x1p96f && vs[0] >= 0x1p-64f && vs[0] <= 0x1p96f;
      k_scales[warp][lane] = good ? ks[0] : 0.f;
      v_log2[warp][lane] = good ? __log2f(vs[0]) : -INFINITY;
      v_inverse[warp][lane] = good ? __fdividef(1.f, vs[0]) : 0.f;
      out = __ballot_sync(0xffffffffu, i < count && has[0] && !good);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
    const uint32_t k_tile = ring + slot * C::kStageBytes, v_tile = k_tile + C::kHalfBytes;
    if (out) {
      // Keys without a scale may hold anything: their rows become zeros.
      if (lane == 0) atomicOr(&bits, DDTREE_ST_BAD_SCALE);
      for (; out; out &= out - 1) {
        const int key = __ffs(out) - 1;
        if (lane < kChunks) {
          asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(k_tile + k_at<kCols>(key, lane)), "r"(0) : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(v_tile + v_at<kCols>(key, lane)), "r"(0) : "memory");
        }
      }
      __syncwarp();
    }
    const uint32_t k_first = k_lane + slot * C::kStageBytes, v_first = v_lane + slot * C::kStageBytes;
    // ---- scores
    float s[kGroups][4];
#pragma unroll
    for (int x = 0; x < kGroups; ++x) s[x][0] = s[x][1] = s[x][2] = s[x][3] = 0.f;
#pragma unroll
    for (int b = 0; b < kCols / 64; ++b) {
#pragma unroll
      for (int x = 0; x < kGroups; ++x) {
        const uint4 codes = lds128((k_first ^ b << 6) + 8 * x * kCols);
        const uint32_t c[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t lo, hi;
          from_codes(c[e], lo, hi);
          mma(s[x], qf[4 * b + e], lo, hi);
        }
      }
    }
    if constexpr (C::kHalves == 2) {
      // The pair's halves add up, through where this tile's K was.
      float4* here = reinterpret_cast<float4*>(smem + (warp * kStages + slot) * C::kStageBytes) + lane;
      const float4* there = here + (half ? -1 : 1) * (kStages * C::kStageBytes / 16);
      __syncwarp();
#pragma unroll
      for (int x = 0; x < kGroups; ++x) here[32 * x] = make_float4(s[x][0], s[x][1], s[x][2], s[x][3]);
      pair_of_warps();
#pragma unroll
      for (int x = 0; x < kGroups; ++x) {
        const float4 v = there[32 * x];
        s[x][0] += v.x; s[x][1] += v.y; s[x][2] += v.z; s[x][3] += v.w;
      }
    }
    // ---- weights: scores in base 2 plus log2 of the value's scale
    uint64_t y[kGroups][2], inv[kGroups];  // keys 2 q4 and 2 q4 + 1 of every eight, of both rows
    const uint64_t by0 = pair(factor[0], factor[0]), by1 = pair(factor[1], factor[1]);
    float high[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int x = 0; x < kGroups; ++x) {
      const uint64_t kf = *reinterpret_cast<const uint64_t*>(&k_scales[warp][8 * x + 2 * q4]);
      const uint64_t vf = *reinterpret_cast<const uint64_t*>(&v_log2[warp][8 * x + 2 * q4]);
      inv[x] = *reinterpret_cast<const uint64_t*>(&v_inverse[warp][8 * x + 2 * q4]);
      y[x][0] = fma2(mul2(pair(s[x][0], s[x][1]), by0), kf, vf);
      y[x][1] = fma2(mul2(pair(s[x][2], s[x][3]), by1), kf, vf);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float2 v = apart(y[x][r]);
        high[r] = max3(high[r], v.x, v.y);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      high[r] = fmaxf(high[r], __shfl_xor_sync(0xffffffffu, high[r], 1));
      high[r] = fmaxf(high[r], __shfl_xor_sync(0xffffffffu, high[r], 2));
    }
    if (__any_sync(0xffffffffu, high[0] - top[0] > kGrowth || high[1] - top[1] > kGrowth)) {  // also the first finite ones
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float to = fmaxf(high[r], top[r]), keep = top[r] == -INFINITY ? 0.f : power2(top[r] - to);
        sum[r] = mul2(sum[r], pair(keep, keep));
        top[r] = to;
#pragma unroll
        for (int d = 0; d < kTilesN; ++d) {
          o[d][2 * r] *= keep;
          o[d][2 * r + 1] *= keep;
        }
      }
    }
    const float from0 = top[0] == -INFINITY ? 0.f : kShift - top[0], from1 = top[1] == -INFINITY ? 0.f : kShift - top[1];
#pragma unroll
    for (int x = 0; x < kGroups; ++x) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float2 v = apart(add2(y[x][r], r ? pair(from1, from1) : pair(from0, from0)));
        s[x][2 * r] = power2(v.x);
        s[x][2 * r + 1] = power2(v.y);
        sum[r] = fma2(pair(s[x][2 * r], s[x][2 * r + 1]), inv[x], sum[r]);
      }
    }
    // ---- O += P V: sixteen keys an instruction, of which the lane has 2 q4, 2 q4 + 1 and the same plus 8
#pragma unroll
    for (int x = 0; x < kGroups / 2; ++x) {
      const uint32_t p[4] = {pack2<true>(s[2 * x][0], s[2 * x][1]), pack2<true>(s[2 * x][2], s[2 * x][3]),
                             pack2<true>(s[2 * x + 1][0], s[2 * x + 1][1]), pack2<true>(s[2 * x + 1][2], s[2 * x + 1][3])};
      constexpr int kWords4 = kChunkCols / 4;
      uint32_t c[4][kWords4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (kChunkCols == 16) {
          const uint4 v = lds128(v_first + (16 * x + (e & 1) + 8 * (e >> 1)) * kCols);
          c[e][0] = v.x; c[e][1] = v.y; c[e][2] = v.z; c[e][3] = v.w;
        } else {
          const uint2 v = lds64((v_first ^ (e & 1) << 6) + (16 * x + 8 * (e >> 1)) * kCols);
          c[e][0] = v.x; c[e][1] = v.y;
        }
      }
#pragma unroll
      for (int w = 0; w < kWords4; ++w) {
        uint32_t b0[4], b1[4];
        from_codes(__byte_perm(c[0][w], c[1][w], 0x5140), b0[0], b0[1]);
        from_codes(__byte_perm(c[0][w], c[1][w], 0x7362), b0[2], b0[3]);
        from_codes(__byte_perm(c[2][w], c[3][w], 0x5140), b1[0], b1[1]);
        from_codes(__byte_perm(c[2][w], c[3][w], 0x7362), b1[2], b1[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) mma(o[4 * w + e], p, b0[e], b1[e]);
      }
    }
    if (joins) {
      // ---- the unit or a chain ends here: the warps' rows are joined through this tile's stages
      const bool whole = unit_ends && !begun;
      const int64_t piece = 2 * share + (begun ? 0 : 1);
      // The unit's record, where it starts; without units' own, the share's, where the share ends.
      if (tid == 0 && last && (unit_records ? !begun : i + 1 == count)) {
        Record r;
        r.token = !unit_ends && !begun ? token : -1;
        r.head = head;
        r.first_share = share;
        const int64_t final_tile = end - 1 + (now.tiles - 1 - tile);  // the unit's last tile in the list
        const int64_t in_longer = longer * (base + 1);
        r.last_share =
            (int)(final_tile < in_longer ? final_tile / (base + 1) : longer + (final_tile - in_longer) / base) * (1 << a.bundle_log2) + sub;
        records[unit_records ? token * a.unit_heads + head : share] = r;
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float2 both = apart(sum[r]);
        float l = both.x + both.y;
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (q4 == 0 && half == 0) {
          top_s[part][g + 8 * r] = top[r];
          sum_s[part][g + 8 * r] = l;
        }
      }
      constexpr int kVecs = kCols / 4;
      // The exchange keeps the rows and columns that eight lanes write at once on other banks.
      auto cell = [&](int w, int r, int c4) {
        return reinterpret_cast<float4*>(smem + (w * kStages + slot) * C::kStageBytes) + r * kVecs + (c4 ^ ((r ^ ((c4 >> 3) << 1)) & 7));
      };
      if constexpr (C::kHalves == 2) pair_of_warps();  // the other one has read the scores
      else __syncwarp();
      // A lane has the columns 2 q4 kChunkCols ..., twice kChunkCols of them.
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (g + 8 * r >= rows) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int t = 0; t < kChunkCols; t += 4)
            *cell(warp, g + 8 * r, ((2 * q4 + h) * kChunkCols + t) / 4) =
                make_float4(o[t][2 * r + h], o[t + 1][2 * r + h], o[t + 2][2 * r + h], o[t + 3][2 * r + h]);
        }
      }
      all_warps();
      for (int e = tid; e < rows * (kDim / 4); e += kThreads) {
        const int row = e / (kDim / 4), vec = e - row * (kDim / 4), col = 4 * vec;
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int k = 0; k < C::kParts; ++k) m = fmaxf(m, top_s[k][row]);
        const float ref = m == -INFINITY ? 0.f : m;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < C::kParts; ++k) {
          const float w = power2(top_s[k][row] - ref);
          const float4 u = *cell(k * C::kHalves + vec / kVecs, row, vec % kVecs);
          l += w * sum_s[k][row];
          x.x += w * u.x; x.y += w * u.y; x.z += w * u.z; x.w += w * u.w;
        }
        if (kLong && (held || !last)) {
          // A long unit's sums so far, the same thread's each time but for the pair.
          float2* pairs = reinterpret_cast<float2*>(a.ws + ws.held_sums) + (int64_t)share * 2 * kRows + row;
          float4* at = reinterpret_cast<float4*>(a.ws + ws.held_rows) + ((int64_t)share * kRows + row) * (kDim / 4) + vec;
          if (held) {
            const float2 s = pairs[(held & 1) * kRows];
            const float4 u = *at;
            const float high = fmaxf(m, s.x), from = high == -INFINITY ? 0.f : high, w = power2(m - from), v = power2(s.x - from);
            m = high;
            l = w * l + v * s.y;
            x.x = w * x.x + v * u.x; x.y = w * x.y + v * u.y; x.z = w * x.z + v * u.z; x.w = w * x.w + v * u.w;
          }
          if (!last) {
            *at = x;
            if (col == 0) pairs[(held + 1 & 1) * kRows] = make_float2(m, l);
            continue;
          }
        }
        if (whole) {
          const float by = l == 0.f ? 0.f : 1.f / l;
          *reinterpret_cast<uint2*>(a.out + token * a.out_stride + (int64_t)(head0 + row) * kDim + col) =
              make_uint2(pack2<kHalf>(x.x * by, x.y * by), pack2<kHalf>(x.z * by, x.w * by));
          if (a.lse && col == 0)
            a.lse[(int64_t)token * a.n_heads + head0 + row] = l == 0.f ? -INFINITY : (m - kShift + log2f(l)) * 0.6931471805599453f;
        } else {
          reinterpret_cast<float4*>(a.ws + ws.rows)[(piece * kRows + row) * (kDim / 4) + vec] = x;
          if (col == 0) reinterpret_cast<float2*>(a.ws + ws.sums)[piece * kRows + row] = make_float2(m, l);
        }
      }
      all_warps();  // the stages are free again
      chain = 0;
      held = last ? 0 : held + 1;
    }
    // ---- the next tile of this stage
    if constexpr (C::kHalves == 2) {
      if (!joins) pair_of_warps();  // the other one has read the scores
    }
#pragma unroll
    for (int k = 0; k + 1 < kStages; ++k) {
      ks[k] = ks[k + 1];
      vs[k] = vs[k + 1];
      has[k] = has[k + 1];
    }
    if (i + kStages < count) start(slot);
    commit();
    if (i + kStages + 1 < count) find();
    // ---- and the tile after this one
    first = joins;
    if (unit_ends) {
      tile = 0;
      begun = false;
      head += 1 << a.bundle_log2;
      if (head >= a.unit_heads && i + 1 < count) {
        head = sub;
        do {
          now = token_of(a, ++token, C::kKeys);
        } while (now.tiles == 0);
      }
    } else {
      ++tile;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  if (tid == 0) words[share] = bits;
}

// Joins the parts of the units that go on across shares: a CTA per record (x),
// slice of its rows (y) and kSplit-th of the columns (z); one more x gathers the
// status words.  kTeams teams of kDim / 4 / kSplit threads, a float4 each, take rows
// of their own, or several share a row's parts; every team keeps its own running
// maximum, so sums and rows are loaded together.  Few records have many parts
// each, and more CTAs (kSplit) load them.
template <bool kHalf, int kDim, int kSplit>
__global__ void __launch_bounds__(256) draft8_join_kernel(const __grid_constant__ Draft8AttnArgs a, int slice_rows) {
  constexpr int kLanes = kDim / 4 / kSplit, kTeams = 256 / kLanes, kTogether = 8;
  __shared__ float4 acc[kTeams][kLanes];
  __shared__ float2 team_sum[kTeams];
  __shared__ uint32_t all;
  const int tid = threadIdx.x;
  const Layout ws = layout_of(kDim, a.n_shares);
  const int x = blockIdx.x, slice = blockIdx.y;
  const int records = by_unit(a) ? a.n_tokens * a.unit_heads : a.n_shares;
  await_grid();
  if (x == records) {
    if (slice > 0 || blockIdx.z > 0) return;
    uint32_t b = 0;
    for (int s = tid; s < a.n_shares; s += 256) b |= reinterpret_cast<const uint32_t*>(a.ws + ws.words)[s];
    if (tid == 0) all = 0;
    __syncthreads();
    if (b) atomicOr(&all, b);
    __syncthreads();
    if (tid == 0) *reinterpret_cast<uint32_t*>(a.ws) = all;
    return;
  }
  // A padding token's units are in no share and nobody wrote their records; what
  // lies there is loaded and dropped.  Bounds hold for every record that was written.
  const Record r = reinterpret_cast<const Record*>(a.ws + ws.records)[x];
  const bool padding = by_unit(a) && __ldg(a.positions + x / a.unit_heads) == -1;
  if (padding || r.token < 0 || r.token >= a.n_tokens || r.head < 0 || r.head >= a.unit_heads || r.first_share < 0 ||
      r.last_share < r.first_share || r.last_share >= a.n_shares)
    return;
  int rows_here;
  const int head = first_head(a, r.head, rows_here);
  const int first = r.first_share, parts = ((r.last_share - first) >> a.bundle_log2) + 1;
  const float2* sums = reinterpret_cast<const float2*>(a.ws + ws.sums);
  const float4* rows = reinterpret_cast<const float4*>(a.ws + ws.rows);
  // Part p of the unit, in every bundle-th share: the second place of the first one, the first place of the others.
  auto place = [&](int p, int row) { return ((int64_t)2 * (first + (p << a.bundle_log2)) + (p == 0)) * kRows + row; };
  const int team = tid / kLanes, lane = tid - team * kLanes, c = blockIdx.z * kLanes + lane;
  const int row_begin = slice * slice_rows, row_end = min(row_begin + slice_rows, rows_here);
  // Teams of a row: as many as the CTA's rows leave, where it has more parts than one team loads at once.
  int per_row = 1;
  while (parts > per_row * kTogether && 2 * per_row * slice_rows <= kTeams) per_row *= 2;
  for (int row0 = row_begin; row0 < row_end; row0 += kTeams / per_row) {
    const int row = row0 + team / per_row;
    float high = -INFINITY, total = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = team % per_row; p0 < parts && row < row_end; p0 += per_row * kTogether) {
      float2 s[kTogether];
      float4 v[kTogether];
#pragma unroll
      for (int u = 0; u < kTogether; ++u) {
        const int p = p0 + u * per_row;
        s[u] = make_float2(-INFINITY, 0.f);
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p < parts) {
          s[u] = sums[place(p, row)];
          v[u] = rows[place(p, row) * (kDim / 4) + c];
        }
      }
      float top = high;
#pragma unroll
      for (int u = 0; u < kTogether; ++u) top = fmaxf(top, s[u].x);
      const float from = top == -INFINITY ? 0.f : top, keep = power2(high - from);
      total *= keep;
      o.x *= keep; o.y *= keep; o.z *= keep; o.w *= keep;
      high = top;
#pragma unroll
      for (int u = 0; u < kTogether; ++u) {
        const float w = power2(s[u].x - from);
        total += w * s[u].y;
        o.x += w * v[u].x; o.y += w * v[u].y; o.z += w * v[u].z; o.w += w * v[u].w;
      }
    }
    if (per_row > 1) {  // the same in the whole CTA
      acc[team][lane] = o;
      if (lane == 0) team_sum[team] = make_float2(high, total);
      __syncthreads();
      if (team % per_row == 0) {
        for (int k = 0; k < per_row; ++k) high = fmaxf(high, team_sum[team + k].x);
        const float from = high == -INFINITY ? 0.f : high;
        o = make_float4(0.f, 0.f, 0.f, 0.f);
        total = 0.f;
        for (int k = 0; k < per_row; ++k) {
          const float w = power2(team_sum[team + k].x - from);
          const float4 v = acc[team + k][lane];
          total += w * team_sum[team + k].y;
          o.x += w * v.x; o.y += w * v.y; o.z += w * v.z; o.w += w * v.w;
        }
      }
      __syncthreads();
    }
    if (team % per_row == 0 && row < row_end) {
      const float by = total == 0.f ? 0.f : 1.f / total;
      *reinterpret_cast<uint2*>(a.out + r.token * a.out_stride + (int64_t)(head + row) * kDim + 4 * c) =
          make_uint2(pack2<kHalf>(o.x * by, o.y * by), pack2<kHalf>(o.z * by, o.w * by));
      if (a.lse && c == 0)
        a.lse[(int64_t)r.token * a.n_heads + head + row] = total == 0.f ? -INFINITY : (high - kShift + log2f(total)) * 0.6931471805599453f;
    }
  }
}

template <bool kHalf, int kDim, bool kLong>
cudaError_t launch_form(const Draft8AttnArgs& a, cudaStream_t stream) {
  using C = Config<kDim>;
  // The shared-memory limit belongs to the kernel on a device: set once on each.
  static std::atomic<uint64_t> have{0};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (device & 63);
  if (!(have.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(draft8_attn_kernel<kHalf, kDim, kLong>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    have.fetch_or(bit, std::memory_order_release);
  }
  e = launch_early(draft8_attn_kernel<kHalf, kDim, kLong>, a.n_shares, kThreads, C::kSmem, stream, a);
  if (e != cudaSuccess) return e;
  // Rows get CTAs of their own where records are few, for their units may have many
  // parts, and where they may have 64, a row's columns too: 185k single, 2 x 256
  // columns, 51.9 -> 46.1 us.  How many there are depends on lengths, which are on the
  // device, so the rule goes by the units: one request of 1 or 2 key heads of 128
  // columns loses 0.3 to 0.5 us by it with a window of 2,048 (7.4 -> 7.7 to 8.0), none
  // with 8,192 (8.6 and 9.0 -> 8.3 and 8.9), and gains at 65,536 keys (16.6 and 15.6 ->
  // 12.4 and 13.5); 256 columns gain from 2,048 keys on.
  const int records = by_unit(a) ? a.n_tokens * a.unit_heads : a.n_shares;
  const int rows = std::min(kRows, a.group);
  const int slices = std::max(1, std::min(rows, a.n_shares / records));
  const int slice_rows = (rows + slices - 1) / slices, slice_count = (rows + slice_rows - 1) / slice_rows;
  constexpr int kSplit = kDim / 32;  // 128 bytes of a row
  if (64 * records <= a.n_shares && (int64_t)records * slice_count * kSplit <= a.n_shares)
    return launch_early(draft8_join_kernel<kHalf, kDim, kSplit>, dim3(records + 1, slice_count, kSplit), 256, 0, stream, a, slice_rows);
  return launch_early(draft8_join_kernel<kHalf, kDim, 1>, dim3(records + 1, slice_count, 1), 256, 0, stream, a, slice_rows);
}

template <bool kHalf, int kDim>
cudaError_t launch(const Draft8AttnArgs& a, cudaStream_t stream) {
  const int64_t of_table = (int64_t)a.table_stride * a.page_size;
  const int64_t keys = a.window > 0 ? std::min(of_table, (int64_t)a.window + a.n_sinks) : of_table;
  return keys > (int64_t)kChain * Config<kDim>::kKeys ? launch_form<kHalf, kDim, true>(a, stream) : launch_form<kHalf, kDim, false>(a, stream);
}

template <bool kHalf>
cudaError_t launch_dim(const Draft8AttnArgs& a, cudaStream_t stream) {
  return a.head_dim == 64 ? launch<kHalf, 64>(a, stream) : a.head_dim == 128 ? launch<kHalf, 128>(a, stream) : launch<kHalf, 256>(a, stream);
}

}  // namespace

static_assert(Config<256>::kCtas == Config<128>::kCtas && Config<64>::kKeys == Config<128>::kKeys, "below");

int draft8_tile_keys(int head_dim) { return head_dim == 256 ? Config<256>::kKeys : Config<128>::kKeys; }

int draft8_shares(int head_dim, int num_sms) {
  return num_sms * (head_dim == 64 ? Config<64>::kCtas : Config<128>::kCtas);
}

int64_t draft8_workspace_bytes(int head_dim, int n_shares) { return (layout_of(head_dim, n_shares).total + 255) / 256 * 256; }

cudaError_t launch_draft8_attention(const Draft8AttnArgs& a, cudaStream_t stream) {
  return a.dtype == DDTREE_FP16 ? launch_dim<true>(a, stream) : launch_dim<false>(a, stream);
}

}  // namespace ddtree
