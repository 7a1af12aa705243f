// The drafter's attention of one new token per request over its cache in 8 bits
// (include/ddtree_draft8.h).
//
//   s_j = scale ks_j <q, kc_j>,  out = sum_j e^(s_j - m) vs_j vc_j / sum_j e^(s_j - m)
//
// with codes kc, vc and their blocks' scales ks, vs.  As with 16 bits the work
// is a stream of keys, and HBM the bound; half the bytes a key leave an SM half
// the time for its arithmetic.  What carries it:
//
//  - The list of tiles, the equal shares, the lookup warp and the join of units
//    that cross shares are those of the 16-bit kernel (k_draft_attn.cu).  Groups
//    of more than 16 query heads are several units of 16, side by side in the list,
//    which read the same keys at the same time.
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
//    So what is rounded to fp16 is a row's weight in the result, at most 1 times
//    a factor of 2^14, whatever the scales are.  A key that is not there has
//    ks = 0, log2 vs = -inf and 1 / vs = 0, and needs no mask.
#include <atomic>

#include "rope.cuh"
#include "tc_ptx.cuh"

namespace ddtree {
namespace {

__host__ __device__ constexpr int keys_of(int dim) { return dim == 64 ? 128 : 64; }
__host__ __device__ constexpr int ctas_of(int dim) { return dim == 256 ? 1 : 2; }
constexpr int kRows = 16;       // query heads of a unit
constexpr float kShift = 14.f;  // log2 of the factor of a probability in fp16

template <int kDim>
struct Config {
  static constexpr int kKeys = keys_of(kDim);
  static constexpr int kWK = 4;                         // warps along the keys of a tile
  static constexpr int kWN = kDim == 256 ? 2 : 1;       // warps along the columns of V (all take the scores)
  static constexpr int kThreads = 32 * kWK * kWN;       // that compute
  static constexpr int kAllThreads = kThreads + 32;
  static constexpr int kStages = kDim == 256 ? 5 : 4;
  static constexpr int kTileBytes = kKeys * kDim;       // of K, and of V
  static constexpr int kQBytes = kRows * kDim * 2;
  static constexpr int kSmem = kStages * (2 * kTileBytes + kQBytes);
  static constexpr int kTileRing = kStages + 2;
  static constexpr int kCols = kDim / kWN;              // columns of a warp
  // The warps' rows are joined in the stage just consumed, so many columns at a time.
  static constexpr int kJoinCols = 2 * kTileBytes / (kWK * kRows * 4) < kDim ? 2 * kTileBytes / (kWK * kRows * 4) : kDim;
};

// A unit that goes on from one share to others: where its parts lie (a record
// per unit where units are no more than shares, else one per share, for the unit
// that starts there and goes on; token -1: nothing to join).
struct Record {
  int32_t token, head, first_share, last_share;
};
__host__ __device__ inline bool by_unit(const Draft8AttnArgs& a) { return (int64_t)a.n_tokens * a.unit_heads <= a.n_shares; }

// Workspace: status block, per share a status word and a record, then the
// (maximum, sum) pairs and the rows of two partial units per share.
struct Layout {
  int64_t words, records, sums, rows, total;
};
__host__ __device__ inline Layout layout_of(int dim, int shares) {
  Layout l;
  l.words = 256;
  l.records = l.words + ((int64_t)shares * 4 + 255) / 256 * 256;
  l.sums = l.records + ((int64_t)shares * 16 + 255) / 256 * 256;
  l.rows = l.sums + ((int64_t)shares * 2 * kRows * 8 + 255) / 256 * 256;
  l.total = l.rows + (int64_t)shares * 2 * kRows * dim * 4;
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

struct Tile {
  int32_t token, head;  // head: of the list, key head and 16 of its query heads
  int32_t unit;         // ordinal within the share: its queries' place
  int32_t flags;
};
enum { kFirst = 1, kLast = 2, kBegun = 4, kGoesOn = 8 };

// Query heads of a unit: the first one, and how many.
__device__ __forceinline__ int first_head(const Draft8AttnArgs& a, int head, int& rows) {
  const int kv = head / a.row_tiles, part = head - kv * a.row_tiles;
  rows = min(kRows, a.group - part * kRows);
  return kv * a.group + part * kRows;
}

template <bool kHalf, int kDim>
__global__ void __launch_bounds__(Config<kDim>::kAllThreads, ctas_of(kDim)) draft8_attn_kernel(const __grid_constant__ Draft8AttnArgs a) {
  using C = Config<kDim>;
  constexpr int kThreads = C::kThreads, kLookup = kThreads / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t offsets[C::kStages][C::kKeys];              // byte offset of a key's row, -1: none
  __shared__ __align__(16) float2 scales[C::kStages][C::kKeys];  // scale of K, log2 of that of V
  __shared__ __align__(16) float inverse[C::kStages][C::kKeys];  // 1 / scale of V
  __shared__ uint32_t dropped[C::kStages][C::kKeys / 32];               // keys whose scale is none
  __shared__ Tile tiles[C::kTileRing];
  __shared__ float top_s[C::kWK][kRows], sum_s[C::kWK][kRows];
  __shared__ int64_t warp_sum[C::kAllThreads / 32];
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

  // ---- lookups by a warp of their own, two or four keys a lane, in three steps a
  // tile each: page numbers, then row offsets and the scales' loads, then the scales.
  // Each step's loads are under way until the next tile's turn.
  constexpr int kStages = C::kStages;
  if (warp == kLookup) {
    constexpr int kPerLane = C::kKeys / 32;
    int cur = start_token, unit = 0;
    Token tok = token_of(a, cur, C::kKeys);
    const int first_bundle = (int)((uint64_t)start_at / (uint32_t)tok.tiles);
    int tile = (int)(start_at - (int64_t)first_bundle * tok.tiles);
    int head = (first_bundle << a.bundle_log2) + sub;
    bool begun = tile > 0;
    int next_pos = -1, next_row = 0;  // of the next token, loaded when the current one is entered
    auto fetch_next = [&] {
      if (cur + 1 < a.n_tokens) {
        next_pos = __ldg(a.positions + cur + 1);
        next_row = row_index(a, cur + 1);
      }
    };
    fetch_next();
    struct Look {
      int page[kPerLane], place[kPerLane], kv_head;  // place -1: no such key
      float ks[kPerLane], vs[kPerLane];
      uint32_t have;                                 // a bit per key that has a row
    };
    auto begin_tile = [&](int i, Look& p) {
      p.kv_head = head / a.row_tiles;
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) {
        const int64_t x = (int64_t)tile * C::kKeys + 32 * k + lane;
        p.page[k] = -1;
        p.place[k] = -1;
        if (x < tok.seen) {
          const int j = (int)(x < tok.first ? x : x - tok.first + tok.lo);
          const int number = a.page.quotient(j);
          p.place[k] = j - number * a.page_size;
          p.page[k] = __ldg(a.table + (int64_t)tok.row * a.table_stride + number);
        }
      }
      const bool unit_ends = tile + 1 == tok.tiles, range_ends = i + 1 == count;
      if (lane == 0) {
        Tile t;
        t.token = cur;
        t.head = head;
        t.unit = unit;
        t.flags = (tile == 0 || i == 0 ? kFirst : 0) | (unit_ends || range_ends ? kLast : 0) | (begun ? kBegun : 0) |
                  (unit_ends ? 0 : kGoesOn);
        tiles[i % C::kTileRing] = t;
        if (tok.seen == 0) atomicOr(&bits, DDTREE_ST_BAD_LENGTH);
        // The unit's record, where it starts; without units' own, the share's, where the share ends.
        const bool goes_on = range_ends && !unit_ends && !begun;
        if (unit_records ? !begun && (unit_ends || range_ends) : range_ends) {
          Record r;
          r.token = goes_on ? cur : -1;
          r.head = head;
          r.first_share = share;
          const int64_t last = end - 1 + (tok.tiles - 1 - tile);  // the unit's last tile in the list
          const int64_t in_longer = longer * (base + 1);
          r.last_share = (int)(last < in_longer ? last / (base + 1) : longer + (last - in_longer) / base) * (1 << a.bundle_log2) + sub;
          records[unit_records ? cur * a.unit_heads + head : share] = r;
        }
      }
      if (unit_ends && !range_ends) {
        tile = 0;
        begun = false;
        ++unit;
        head += 1 << a.bundle_log2;
        if (head >= a.unit_heads) {
          head = sub;
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
    auto place_tile = [&](int i, Look& p) {
      p.have = 0;
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) {
        const bool good = p.page[k] >= 0 && p.page[k] < a.n_pages;
        if (p.place[k] >= 0 && !good) atomicOr(&bits, DDTREE_ST_BAD_INDEX);
        offsets[i % kStages][32 * k + lane] =
            good ? p.page[k] * a.page_stride + p.place[k] * a.token_stride + p.kv_head * a.head_stride : -1;
        p.ks[k] = p.vs[k] = 0.f;
        if (good) {
          const int64_t s = ((int64_t)p.page[k] * a.blocks + a.block.quotient(p.place[k])) * a.n_kv_heads + p.kv_head;
          p.ks[k] = a.k_scale[s];
          p.vs[k] = a.v_scale[s];
          p.have |= 1u << k;
        }
      }
    };
    auto scale_tile = [&](int i, const Look& p) {
      const int slot = i % kStages;
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) {
        const bool good = p.ks[k] >= 0x1p-64f && p.ks[k] <= 0x1p96f && p.vs[k] >= 0x1p-64f && p.vs[k] <= 0x1p96f;
        scales[slot][32 * k + lane] = good ? make_float2(p.ks[k], log2f(p.vs[k])) : make_float2(0.f, -INFINITY);
        inverse[slot][32 * k + lane] = good ? 1.f / p.vs[k] : 0.f;
        const uint32_t out = __ballot_sync(0xffffffffu, (p.have >> k & 1) && !good);
        if (lane == 0) {
          dropped[slot][k] = out;
          if (out) atomicOr(&bits, DDTREE_ST_BAD_SCALE);
        }
      }
    };
    Look placed, ahead;
    {
      Look first[kStages];
#pragma unroll
      for (int i = 0; i < kStages; ++i)
        if (i < count) begin_tile(i, first[i]);
#pragma unroll
      for (int i = 0; i < kStages; ++i)
        if (i < count) place_tile(i, first[i]);
      if (kStages < count) begin_tile(kStages, ahead);
      __syncthreads();  // the copies of tiles 0 .. kStages - 2 may start
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i)
        if (i < count) scale_tile(i, first[i]);
      placed = first[kStages - 1];
    }
    for (int i = 0; i < count; ++i) {
      __syncthreads();  // tile i is computed, the copies of tile i + kStages - 1 start
      if (i + kStages - 1 < count) scale_tile(i + kStages - 1, placed);
      if (i + kStages < count) {
        place_tile(i + kStages, ahead);
        placed = ahead;
      }
      if (i + kStages + 1 < count) begin_tile(i + kStages + 1, ahead);
    }
    __syncthreads();
    if (lane == 0) words[share] = bits;
    return;
  }

  // ---- copies: a thread has one 16-byte chunk of every kRowsPerStep-th key
  const uint32_t ring = ptx::smem_u32(smem), q_ring = ring + kStages * 2 * C::kTileBytes;
  constexpr int kChunks = kDim / 16, kRowsPerStep = kThreads / kChunks;
  static_assert(C::kKeys % kRowsPerStep == 0 && kRowsPerStep % 8 == 0, "copy steps");
  const int copy_chunk = tid % kChunks, copy_row = tid / kChunks;
  // Steps of eight rows leave the exchange of chunks as it is.
  const uint32_t copy_k = k_at<kDim>(copy_row, copy_chunk), copy_v = C::kTileBytes + v_at<kDim>(copy_row, copy_chunk);
  const uint8_t *k_src = a.k + 16 * copy_chunk, *v_src = a.v + 16 * copy_chunk;
  auto start_copies = [&](int i) {
    if (i < count) {
      const uint32_t stage = ring + (i % kStages) * 2 * C::kTileBytes;
#pragma unroll
      for (int r = 0; r < C::kKeys; r += kRowsPerStep) {
        const int64_t off = offsets[i % kStages][copy_row + r];
        const uint32_t size = off < 0 ? 0u : 16u;
        ptx::cp_async16_zfill(stage + copy_k + r * kDim, k_src + (off < 0 ? 0 : off), size);
        ptx::cp_async16_zfill(stage + copy_v + r * kDim, v_src + (off < 0 ? 0 : off), size);
      }
      const Tile t = tiles[i % C::kTileRing];
      if (t.flags & kFirst) {
        int rows;
        const uint16_t* q = a.q + t.token * a.q_stride + (int64_t)first_head(a, t.head, rows) * kDim;
        const uint32_t q_at = q_ring + (t.unit % kStages) * C::kQBytes;
#pragma unroll
        for (int e = tid; e < kRows * (kDim / 8); e += kThreads) {
          const int r = e / (kDim / 8);
          ptx::cp_async16_zfill(q_at + e * 16, r < rows ? q + e * 8 : a.q, r < rows ? 16u : 0u);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) start_copies(i);

  auto computing_warps = [] { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); };
  // ---- this warp's keys of every tile, and its columns of V
  const int wn = warp % C::kWN, wk = warp / C::kWN, g = lane >> 2, q4 = lane & 3;
  constexpr int kWarpKeys = C::kKeys / C::kWK, kGroups = kWarpKeys / 8;  // of eight keys
  constexpr int kChunkCols = C::kCols / 8;                               // columns of V that a lane reads: 16 or 8
  constexpr int kTilesN = C::kCols / 8;                                  // product tiles of eight columns
  const int key0 = wk * kWarpKeys;
  uint32_t qf[kDim / 16][4];
  float o[kTilesN][4], top[2], sum[2], factor[2];

  for (int i = 0; i < count; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncthreads();
    start_copies(i + kStages - 1);
    const int slot = i % kStages;
    const Tile t = tiles[i % C::kTileRing];
    const uint32_t k_tile = ring + slot * 2 * C::kTileBytes, v_tile = k_tile + C::kTileBytes;
    if (t.flags & kFirst) {
      // Columns 16 q4 .. 16 q4 + 15 of every 64, of rows g and g + 8: four of them an instruction.
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t q_at = q_ring + (t.unit % kStages) * C::kQBytes + (g + 8 * r) * kDim * 2 + q4 * 32;
        float most = 0.f;
#pragma unroll
        for (int b = 0; b < kDim / 32; ++b) {
          const uint4 v = lds128(q_at + (b >> 1) * 128 + (b & 1) * 16);
          float x[8];
          unpack8<kHalf>(v, x);
#pragma unroll
          for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(x[e]));
        }
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        // The largest element to [2^14, 2^15).
        const int up = most == 0.f ? 0 : max(-110, min(120, 14 + 127 - (int)(__float_as_uint(most) >> 23)));
        const float by = __uint_as_float((uint32_t)(up + 127) << 23);
        factor[r] = __uint_as_float((uint32_t)(127 - up) << 23) * a.scale_log2;
#pragma unroll
        for (int b = 0; b < kDim / 32; ++b) {
          const uint4 v = lds128(q_at + (b >> 1) * 128 + (b & 1) * 16);
          float x[8];
          unpack8<kHalf>(v, x);
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
      sum[0] = sum[1] = 0.f;
    }
    // Keys without a scale may hold anything: their rows become zeros.
    uint32_t out = dropped[slot][key0 >> 5] >> (key0 & 31) & (kWarpKeys == 32 ? 0xffffffffu : (1u << (kWarpKeys & 31)) - 1);
    if (out) {
      for (; out; out &= out - 1) {
        const int key = key0 + __ffs(out) - 1;
        if (lane < kChunks) {
          asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(k_tile + k_at<kDim>(key, lane)), "r"(0) : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(v_tile + v_at<kDim>(key, lane)), "r"(0) : "memory");
        }
      }
      __syncwarp();
    }
    // ---- scores
    float s[kGroups][4];
#pragma unroll
    for (int x = 0; x < kGroups; ++x) s[x][0] = s[x][1] = s[x][2] = s[x][3] = 0.f;
#pragma unroll
    for (int b = 0; b < kDim / 64; ++b) {
#pragma unroll
      for (int x = 0; x < kGroups; ++x) {
        const uint4 codes = lds128(k_tile + k_at<kDim>(key0 + 8 * x + g, 4 * b + q4));
        const uint32_t c[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t lo, hi;
          from_codes(c[e], lo, hi);
          mma(s[x], qf[4 * b + e], lo, hi);
        }
      }
    }
    // ---- weights: scores in base 2 plus log2 of the value's scale
    float inv[kGroups][2], high[2] = {top[0], top[1]};
#pragma unroll
    for (int x = 0; x < kGroups; ++x) {
      const float4 f = *reinterpret_cast<const float4*>(&scales[slot][key0 + 8 * x + 2 * q4]);
      const float2 w = *reinterpret_cast<const float2*>(&inverse[slot][key0 + 8 * x + 2 * q4]);
      inv[x][0] = w.x;
      inv[x][1] = w.y;
      s[x][0] = fmaf(s[x][0] * factor[0], f.x, f.y);
      s[x][1] = fmaf(s[x][1] * factor[0], f.z, f.w);
      s[x][2] = fmaf(s[x][2] * factor[1], f.x, f.y);
      s[x][3] = fmaf(s[x][3] * factor[1], f.z, f.w);
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
        const float keep = top[r] == -INFINITY ? 0.f : power2(top[r] - high[r]);
        sum[r] *= keep;
        top[r] = high[r];
#pragma unroll
        for (int d = 0; d < kTilesN; ++d) {
          o[d][2 * r] *= keep;
          o[d][2 * r + 1] *= keep;
        }
      }
    }
    const float from[2] = {top[0] == -INFINITY ? 0.f : kShift - top[0], top[1] == -INFINITY ? 0.f : kShift - top[1]};
#pragma unroll
    for (int x = 0; x < kGroups; ++x) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[x][e] = power2(s[x][e] + from[e >> 1]);
        sum[e >> 1] = fmaf(s[x][e], inv[x][e & 1], sum[e >> 1]);
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
        const int key = key0 + 16 * x + 2 * q4 + (e & 1) + 8 * (e >> 1);
        if constexpr (kChunkCols == 16) {
          const uint4 v = lds128(v_tile + v_at<kDim>(key, wn * 8 + g));
          c[e][0] = v.x; c[e][1] = v.y; c[e][2] = v.z; c[e][3] = v.w;
        } else {
          const uint2 v = lds64(v_tile + v_at<kDim>(key, g >> 1) + (g & 1) * 8);
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
    if (!(t.flags & kLast)) continue;

    // ---- the unit ends here: the warps' rows are joined through this tile's stage
    const bool whole = !(t.flags & (kBegun | kGoesOn));
    const int64_t part = 2 * share + (t.flags & kBegun ? 0 : 1);
    int rows;
    const int head = first_head(a, t.head, rows);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
      sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
      if (q4 == 0 && wn == 0) {
        top_s[wk][g + 8 * r] = top[r];
        sum_s[wk][g + 8 * r] = sum[r];
      }
    }
    float4* buffer = reinterpret_cast<float4*>(smem + slot * 2 * C::kTileBytes);
    constexpr int kVecs = C::kJoinCols / 4;
    // The exchange keeps the rows and columns that eight lanes write at once on other banks.
    auto cell = [&](int w, int r, int c4) { return buffer + (w * kRows + r) * kVecs + (c4 ^ ((r ^ ((c4 >> 3) << 1)) & 7)); };
#pragma unroll
    for (int pass = 0; pass < kDim / C::kJoinCols; ++pass) {
      computing_warps();  // the stage is free: every warp is done with the tile, or with the last columns
      // A lane has columns wn kCols + 2 q4 kChunkCols ... twice kChunkCols of them.
      const int col0 = wn * C::kCols + 2 * q4 * kChunkCols - pass * C::kJoinCols;
      if (col0 >= 0 && col0 < C::kJoinCols) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (g + 8 * r >= rows) continue;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int d = 0; d < kChunkCols / 4; ++d)
              *cell(wk, g + 8 * r, (col0 + h * kChunkCols) / 4 + d) =
                  make_float4(o[4 * d][2 * r + h], o[4 * d + 1][2 * r + h], o[4 * d + 2][2 * r + h], o[4 * d + 3][2 * r + h]);
          }
        }
      }
      computing_warps();
      for (int e = tid; e < rows * kVecs; e += kThreads) {
        const int row = e / kVecs, c4 = e - row * kVecs, col = pass * C::kJoinCols + 4 * c4;
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int k = 0; k < C::kWK; ++k) m = fmaxf(m, top_s[k][row]);
        const float ref = m == -INFINITY ? 0.f : m;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < C::kWK; ++k) {
          const float w = power2(top_s[k][row] - ref);
          const float4 u = *cell(k, row, c4);
          l += w * sum_s[k][row];
          x.x += w * u.x; x.y += w * u.y; x.z += w * u.z; x.w += w * u.w;
        }
        if (whole) {
          const float by = l == 0.f ? 0.f : 1.f / l;
          *reinterpret_cast<uint2*>(a.out + t.token * a.out_stride + (int64_t)(head + row) * kDim + col) =
              make_uint2(pack2<kHalf>(x.x * by, x.y * by), pack2<kHalf>(x.z * by, x.w * by));
          if (a.lse && col == 0)
            a.lse[(int64_t)t.token * a.n_heads + head + row] = l == 0.f ? -INFINITY : (m - kShift + log2f(l)) * 0.6931471805599453f;
        } else {
          reinterpret_cast<float4*>(a.ws + ws.rows)[(part * kRows + row) * (kDim / 4) + col / 4] = x;
          if (col == 0) reinterpret_cast<float2*>(a.ws + ws.sums)[part * kRows + row] = make_float2(m, l);
        }
      }
    }
    // The next iteration's barrier comes before this stage is filled again.
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
}

// Joins the parts of the units that go on across shares, as the 16-bit kernel's
// join does: a CTA per record (x) and slice of its rows (y); one more x gathers
// the status words.  Eight teams of kDim / 4 threads take rows of their own, or
// several share a row's parts.
template <bool kHalf, int kDim>
__global__ void __launch_bounds__(2 * kDim) draft8_join_kernel(const __grid_constant__ Draft8AttnArgs a, int slice_rows) {
  constexpr int kTeams = 8, kLanes = kDim / 4, kTogether = 8;
  constexpr int kThreads = kTeams * kLanes;
  __shared__ float4 acc[kTeams][kLanes];
  __shared__ float2 team_sum[kTeams];
  __shared__ uint32_t all;
  const int tid = threadIdx.x;
  const Layout ws = layout_of(kDim, a.n_shares);
  const int x = blockIdx.x, slice = blockIdx.y;
  const int records = by_unit(a) ? a.n_tokens * a.unit_heads : a.n_shares;
  await_grid();
  if (x == records) {
    if (slice > 0) return;
    uint32_t b = 0;
    for (int s = tid; s < a.n_shares; s += kThreads) b |= reinterpret_cast<const uint32_t*>(a.ws + ws.words)[s];
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
  const int team = tid / kLanes, c = tid - team * kLanes;
  const int row_begin = slice * slice_rows, row_end = min(row_begin + slice_rows, rows_here);
  const int per_row = parts <= kTogether || slice_rows > 4 ? 1 : slice_rows > 2 ? 2 : slice_rows > 1 ? 4 : 8;
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
          v[u] = rows[place(p, row) * kLanes + c];
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
      const float by = total == 0.f ? 0.f : 1.f / total;
      *reinterpret_cast<uint2*>(a.out + r.token * a.out_stride + (int64_t)(head + row) * kDim + 4 * c) =
          make_uint2(pack2<kHalf>(o.x * by, o.y * by), pack2<kHalf>(o.z * by, o.w * by));
      if (a.lse && c == 0)
        a.lse[(int64_t)r.token * a.n_heads + head + row] = total == 0.f ? -INFINITY : (high - kShift + log2f(total)) * 0.6931471805599453f;
    }
  }
}

template <bool kHalf, int kDim>
cudaError_t launch(const Draft8AttnArgs& a, cudaStream_t stream) {
  using C = Config<kDim>;
  // The shared-memory limit belongs to the kernel on a device: set once on each.
  static std::atomic<uint64_t> have{0};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (device & 63);
  if (!(have.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(draft8_attn_kernel<kHalf, kDim>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    have.fetch_or(bit, std::memory_order_release);
  }
  e = launch_early(draft8_attn_kernel<kHalf, kDim>, a.n_shares, C::kAllThreads, C::kSmem, stream, a);
  if (e != cudaSuccess) return e;
  // Rows get CTAs of their own where records are few, for their units have many parts.
  const int records = by_unit(a) ? a.n_tokens * a.unit_heads : a.n_shares;
  const int rows = std::min(kRows, a.group);
  const int slices = std::max(1, std::min(rows, a.n_shares / records));
  const int slice_rows = (rows + slices - 1) / slices;
  return launch_early(draft8_join_kernel<kHalf, kDim>, dim3(records + 1, (rows + slice_rows - 1) / slice_rows), 2 * kDim, 0, stream, a,
                      slice_rows);
}

template <bool kHalf>
cudaError_t launch_dim(const Draft8AttnArgs& a, cudaStream_t stream) {
  return a.head_dim == 64 ? launch<kHalf, 64>(a, stream) : a.head_dim == 128 ? launch<kHalf, 128>(a, stream) : launch<kHalf, 256>(a, stream);
}

}  // namespace

int draft8_tile_keys(int head_dim) { return keys_of(head_dim); }

int draft8_shares(int head_dim, int num_sms) { return ctas_of(head_dim) * num_sms; }

int64_t draft8_workspace_bytes(int head_dim, int n_shares) { return (layout_of(head_dim, n_shares).total + 255) / 256 * 256; }

cudaError_t launch_draft8_attention(const Draft8AttnArgs& a, cudaStream_t stream) {
  return a.dtype == DDTREE_FP16 ? launch_dim<true>(a, stream) : launch_dim<false>(a, stream);
}

}  // namespace ddtree
