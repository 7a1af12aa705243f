// The drafter's new queries, keys and values with a cache in 8 bits
// (include/ddtree_draft8.h): head norms, rotation, quantisation as the rows are
// written; and rows read back.
//
// A CTA takes a chunk of up to eight tokens, or a slice of its heads where tokens are
// few, and puts the sines and cosines of its tokens into shared memory: every row
// of a token needs the same.  Queries go row by row, and so do keys and values
// where every token has scales of its own (blocks of one token).
//
// Keys and values: the rows that a call writes to one block (a run of the list)
// share a scale, which depends on the largest magnitude of them all, so the
// unit of work is a run of one key head.  A team of 1, 2 or 4 warps holds the
// run's up to 4,096 elements in registers as 32-bit numbers (32 a lane): read
// once, rounded once, written once, with one exchange of maxima between.  Runs
// are found where the block changes in the list, by a ballot over a chunk of
// tokens; the warp at a run's first token takes the whole run, also what lies
// behind its chunk.  A block that has to grow moves its other rows to the new
// scale there and then: nobody else writes that block in the call.
//
// To read and write: 2 + 2 bytes a query element, 2 + 1 a key's or value's.  32,749
// tokens of 32 + 8 heads of 128 columns (738 MB): 170 us, 4.3 TB/s, 0.65 of the copy
// rate.  Of some 104 M warp instructions (the issue slots are 55 % busy) norms,
// rotation and conversions are the most, and the next rows' loads have to hide
// behind them in 16 warps an SM: 128 registers hold four rows a lane and the four
// behind them.  With the rows read back as well 203 us; there five CTAs an SM, which
// spill, take 251 and six 274, chunks of 4 and 16 tokens 218 and 211, queries and runs
// as launches of their own 280.  Small calls (8 tokens of the same heads, one for
// each block): 5.3 us in a graph, launch and three loads that wait for each other
// (places, rows and scales, the block's old rows).
#include "../../include/ddtree_draft8.h"
#include "f32x2.cuh"
#include "rope.cuh"

namespace ddtree {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;   // head steps of a query whose loads are in flight together
constexpr int kSteps = 4;    // row steps of a warp in a run

// turn() of the 16-bit appends with the nearest quarter taken off as a whole number,
// so that the rest is off by a quarter as much (2.3e-8 in place of 9.4e-8) when it is
// rounded to 32 bits.  Keys are quantised from 32 bits, and those next to a border
// between two codes tell: of 33.5 million, 40 to 57 fall on the other side of it than
// in 64 bits (71 to 100 with turn(); 48 to 75 with angles in 64 bits and elementary
// 32-bit operations).
__device__ __forceinline__ float2 close_turn(uint64_t f, int32_t position, float mscale) {
  const uint32_t p = (uint32_t)position;
  const uint32_t t = (uint32_t)(f >> 32) * p + __umulhi((uint32_t)f, p);
  const uint32_t quarter = (t + 0x20000000u) >> 30;
  float s, c;
  sincospif((float)(int32_t)(t - (quarter << 30)) * 0x1p-31f, &s, &c);
  const float x = quarter & 1 ? -s : c, y = quarter & 1 ? c : s, m = quarter & 2 ? -mscale : mscale;
  return make_float2(x * m, y * m);
}

__device__ __forceinline__ bool scale_ok(float s) { return s >= 0x1p-64f && s <= 0x1p96f; }

// The least power of two s with top <= 448 s (448 = 1.75 * 2^8); 1 for 0.
__device__ __forceinline__ float scale_for(float top) {
  const uint32_t b = __float_as_uint(top);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u);
  return top == 0.f ? 1.f : __uint_as_float((uint32_t)(max(-64, min(96, e)) + 127) << 23);
}

// Four numbers to e4m3, nearest, ties to even, the largest beyond the range.
__device__ __forceinline__ uint32_t to_codes(float a, float b, float c, float d) {
  uint32_t r;
  asm("{ .reg .b16 lo, hi;\n"
      "  cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n"
      "  cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
      "  mov.b32 %0, {lo, hi}; }"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// Four codes as fp16 pairs (exact).
__device__ __forceinline__ void from_codes(uint32_t c, uint32_t& lo, uint32_t& hi) {
  asm("{ .reg .b16 a, b;\n"
      "  mov.b32 {a, b}, %2;\n"
      "  cvt.rn.f16x2.e4m3x2 %0, a;\n"
      "  cvt.rn.f16x2.e4m3x2 %1, b; }"
      : "=r"(lo), "=r"(hi)
      : "r"(c));
}
__device__ __forceinline__ void unpack_codes8(uint2 c, float (&x)[8]) {
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t lo, hi;
    from_codes(w[i], lo, hi);
    const float2 a = unpack2<true>(lo), b = unpack2<true>(hi);
    x[4 * i] = a.x; x[4 * i + 1] = a.y; x[4 * i + 2] = b.x; x[4 * i + 3] = b.y;
  }
}
// Eight numbers of a row, two by two.
struct Row {
  uint64_t v[4];
};
template <bool kHalf>
__device__ __forceinline__ Row unpack_row(const uint4& in) {
  const uint32_t w[4] = {in.x, in.y, in.z, in.w};
  Row r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = unpack2<kHalf>(w[j]);
    r.v[j] = pair(x.x, x.y);
  }
  return r;
}
template <bool kHalf>
__device__ __forceinline__ uint4 pack_row(const Row& r) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = apart(r.v[j]);
    w[j] = pack2<kHalf>(x.x, x.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// x / s: a product where s is a power of two (also exact), else the quotient.
__device__ __forceinline__ uint2 quantise_row(const Row& r, float s) {
  float2 y[4];
  if ((__float_as_uint(s) & 0x7fffffu) == 0) {
    const float inv = __uint_as_float((254u << 23) - __float_as_uint(s));
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = apart(mul2(r.v[j], pair(inv, inv)));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[j] = apart(r.v[j]);
      y[j] = make_float2(__fdiv_rn(y[j].x, s), __fdiv_rn(y[j].y, s));
    }
  }
  return make_uint2(to_codes(y[0].x, y[0].y, y[1].x, y[1].y), to_codes(y[2].x, y[2].y, y[3].x, y[3].y));
}

// A row lies over kDim / 8 lanes.  A lane has two pieces of four columns: where the
// rotation is on halves the same place of both, so that a pair's elements meet in
// one lane; else (interleaved pairs, columns that are not rotated) eight next to
// each other.
template <int kDim, bool kInterleaved>
struct Lane {
  int a, b;      // first column of each piece
  int pair;      // first of the lane's four pairs
  bool turned;
  __device__ __forceinline__ Lane(int rot_dim, int c) {
    turned = 8 * c < rot_dim;
    pair = turned ? 4 * c : 0;
    a = kInterleaved || !turned ? 8 * c : 4 * c;
    b = kInterleaved || !turned ? 8 * c + 4 : rot_dim / 2 + 4 * c;
  }
  __device__ __forceinline__ uint4 load(const uint16_t* row) const {
    const uint2 u = *reinterpret_cast<const uint2*>(row + a), v = *reinterpret_cast<const uint2*>(row + b);
    return make_uint4(u.x, u.y, v.x, v.y);
  }
  __device__ __forceinline__ void store(uint16_t* row, const uint4& v) const {
    *reinterpret_cast<uint2*>(row + a) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2*>(row + b) = make_uint2(v.z, v.w);
  }
  __device__ __forceinline__ uint2 load_codes(const uint8_t* row) const {
    return make_uint2(*reinterpret_cast<const uint32_t*>(row + a), *reinterpret_cast<const uint32_t*>(row + b));
  }
  __device__ __forceinline__ void store_codes(uint8_t* row, uint2 v) const {
    *reinterpret_cast<uint32_t*>(row + a) = v.x;
    *reinterpret_cast<uint32_t*>(row + b) = v.y;
  }
};

// A token's rotation of a lane's four pairs: v = v * same + other elements of the pairs * across.
template <bool kInterleaved>
struct Turn {
  uint64_t same[4], across[4];
  // cosines and sines of the pairs, one behind the other
  __device__ __forceinline__ Turn(const float* cosines, const float* sines) {
    const float4 c = *reinterpret_cast<const float4*>(cosines), s = *reinterpret_cast<const float4*>(sines);
    if constexpr (kInterleaved) {
      same[0] = pair(c.x, c.x); same[1] = pair(c.y, c.y); same[2] = pair(c.z, c.z); same[3] = pair(c.w, c.w);
      across[0] = pair(-s.x, s.x); across[1] = pair(-s.y, s.y); across[2] = pair(-s.z, s.z); across[3] = pair(-s.w, s.w);
    } else {
      same[0] = same[2] = pair(c.x, c.y);
      same[1] = same[3] = pair(c.z, c.w);
      across[0] = pair(-s.x, -s.y); across[1] = pair(-s.z, -s.w);
      across[2] = pair(s.x, s.y); across[3] = pair(s.z, s.w);
    }
  }
  __device__ __forceinline__ void apply(Row& r) const {
    Row o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (kInterleaved) {
        const float2 x = apart(r.v[j]);
        o.v[j] = pair(x.y, x.x);
      } else {
        o.v[j] = r.v[j ^ 2];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) r.v[j] = fma2(o.v[j], across[j], mul2(r.v[j], same[j]));
  }
};

// 1 / root mean square of rows that kDim / 8 lanes hold each, side by side.
template <int kDim, int kCount>
__device__ __forceinline__ void row_norms(const Row (&r)[kCount], float eps, float (&by)[kCount]) {
#pragma unroll
  for (int i = 0; i < kCount; ++i) {
    const uint64_t* v = r[i].v;
    const float2 s = apart(fma2(v[3], v[3], fma2(v[2], v[2], fma2(v[1], v[1], mul2(v[0], v[0])))));
    by[i] = s.x + s.y;
  }
#pragma unroll
  for (int d = kDim / 16; d > 0; d >>= 1) {
#pragma unroll
    for (int i = 0; i < kCount; ++i) by[i] += __shfl_xor_sync(0xffffffffu, by[i], d);
  }
#pragma unroll
  for (int i = 0; i < kCount; ++i) by[i] = rsqrtf(by[i] * (1.f / kDim) + eps);
}
__device__ __forceinline__ void scale_row(Row& r, float by, const Row& weight) {
#pragma unroll
  for (int j = 0; j < 4; ++j) r.v[j] = mul2(mul2(r.v[j], pair(by, by)), weight.v[j]);
}
// Largest magnitude; NaN is passed over, and so are infinities where kFinite.
template <bool kFinite>
__device__ __forceinline__ float row_top(const Row& r, float top) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = apart(r.v[j]);
    const float a = fabsf(x.x), b = fabsf(x.y);
    if (!kFinite || a < INFINITY) top = fmaxf(top, a);
    if (!kFinite || b < INFINITY) top = fmaxf(top, b);
  }
  return top;
}

// Grid: chunks of `chunk` tokens (a power of two), slices of their heads: the first
// row_slices for rows on their own and the others for runs, or one for both.
// team: warps of a run.  kByRow: every token has its own scale, all rows are on their own.
template <bool kHalf, int kDim, bool kInterleaved, bool kByRow>
__global__ void __launch_bounds__(kThreads, 4) draft8_append_kernel(const __grid_constant__ Draft8AppendArgs a, int chunk, int team, int row_slices) {
  constexpr int kLanes = kDim / 8;        // lanes of a row
  constexpr int kRows = 32 / kLanes;      // rows of a warp's step
  // Of the chunk's tokens, and of those behind it that end its last run: cosines, then sines.
  extern __shared__ __align__(16) float turns[];
  __shared__ float tops[2][kWarps];
  await_grid();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = lane % kLanes, sub = lane / kLanes;
  const Lane<kDim, kInterleaved> mine(a.rope.rot_dim, c);
  const bool both = !kByRow && gridDim.y == 1, rows_on = both || blockIdx.y < row_slices, runs_on = !kByRow && (both || !rows_on);
  const int slice = rows_on ? blockIdx.y : blockIdx.y - row_slices, slices = both ? 1 : rows_on ? row_slices : gridDim.y - row_slices;
  const int n0 = blockIdx.x * chunk, n_end = min(n0 + chunk, a.n_tokens);
  const uint4 none = make_uint4(0, 0, 0, 0);

  // Before a CTA in which no run begins leaves: without queries there may be no other one for its tokens.
  if (blockIdx.y == 0 && warp == 0 && a.status && n0 + lane < n_end) {
    const int pos = __ldg(a.positions + n0 + lane), slot = __ldg(a.slots + n0 + lane);
    if (pos < -1) atomicOr(a.status, DDTREE_ST_BAD_LENGTH);
    else if (pos >= 0 && (slot < -1 || slot >= a.total_slots)) atomicOr(a.status, DDTREE_ST_BAD_INDEX);
  }

  // ---- the chunk's runs: lane i has token n0 + i, and the i-th and i + 32-th behind the chunk
  struct Spot {
    int block, place;  // number of the token's block, its place there; -1 where nothing is written
  };
  auto spot_of = [&](int n) {
    Spot s = {-1, 0};
    if (n < 0 || n >= a.n_tokens) return s;
    const int pos = __ldg(a.positions + n), slot = __ldg(a.slots + n);
    if (pos < 0 || slot < 0 || slot >= a.total_slots) return s;
    const int page = a.page.quotient(slot), in_page = slot - page * a.page_size, b = a.block.quotient(in_page);
    s.block = page * a.blocks + b;
    s.place = in_page - b * a.block_tokens;
    return s;
  };
  Spot here = {-1, 0}, behind[2] = {{-1, 0}, {-1, 0}};
  uint32_t leaders = 0;
  int tail = 0;
  if (runs_on) {
    // All loads at once.
    if (n0 + lane < n_end) here = spot_of(n0 + lane);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (32 * k + lane < a.block_tokens - 1) behind[k] = spot_of(n_end + 32 * k + lane);
    const int first_before = spot_of(n0 - 1).block;
    const int last = __shfl_sync(0xffffffffu, here.block, n_end - 1 - n0);
    uint32_t same[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) same[k] = __ballot_sync(0xffffffffu, last >= 0 && behind[k].block == last);
    tail = ~same[0] ? __ffs(~same[0]) - 1 : ~same[1] ? 31 + __ffs(~same[1]) : 64;
    int before = __shfl_up_sync(0xffffffffu, here.block, 1);
    if (lane == 0) before = first_before;
    leaders = __ballot_sync(0xffffffffu, here.block >= 0 && here.block != before);
    if (!leaders) {
      if (!rows_on) return;  // the whole CTA: nothing begins here
      tail = 0;
    }
  }
  const int pairs = a.rope.rot_dim / 2;
  Row wq = {}, wk = {};
  if (a.q_weight) wq = unpack_row<kHalf>(mine.load(a.q_weight));
  if (kByRow && a.k_weight) wk = unpack_row<kHalf>(mine.load(a.k_weight));

  // ---- rows on their own: a warp has tokens of the chunk, or some heads of one.  A
  // batch is kUnroll steps; the next one, of whatever token, is loaded before this
  // one is computed, and the first one before the sines are ready.
  const int nq = a.n_heads, nk = a.n_kv_heads, heads = kByRow ? nq + 2 * nk : nq;
  const int per_token = chunk < kWarps ? kWarps / chunk : 1;  // warps of a token
  const int row_parts = slices * per_token, part_steps = ((heads + kRows - 1) / kRows + row_parts - 1) / row_parts;
  const int h_begin = (slice * per_token + warp % per_token) * part_steps * kRows, h_end = min(h_begin + part_steps * kRows, heads);
  const int n_step = kWarps / per_token;
  auto load_batch = [&](int n, int h, uint4 (&in)[kUnroll]) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int at = h + u * kRows + sub;
      in[u] = none;
      if (n < n_end && at < h_end) {  // plain loads: q_out may be q
        const uint16_t* src = !kByRow || at < nq ? a.q + n * a.q_stride + at * kDim
                              : at < nq + nk     ? a.k + n * a.k_stride + (at - nq) * kDim
                                                 : a.v + n * a.v_stride + (at - nq - nk) * kDim;
        in[u] = mine.load(src);
      }
    }
  };
  uint4 next[kUnroll];
  int n = rows_on && h_begin < h_end ? n0 + warp / per_token : n_end, h = h_begin;
  load_batch(n, h, next);
  for (int t = warp; t < n_end - n0 + tail; t += kWarps) {
    const int pos = __ldg(a.positions + n0 + t);
    for (int p = lane; p < pairs; p += 32) {
      const float2 cs = close_turn(a.rope.turns[p], pos, a.rope.mscale);
      turns[2 * t * pairs + p] = cs.x;
      turns[(2 * t + 1) * pairs + p] = cs.y;
    }
  }
  __syncthreads();
  while (n < n_end) {
    Row x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) x[u] = unpack_row<kHalf>(next[u]);
    const int n_now = n, h_now = h;
    h += kRows * kUnroll;
    if (h >= h_end) {
      h = h_begin;
      n += n_step;
    }
    load_batch(n, h, next);
    if (__ldg(a.positions + n_now) < 0) continue;
    const float* cs = turns + 2 * (n_now - n0) * pairs + mine.pair;
    const Turn<kInterleaved> rotation(cs, cs + pairs);
    if constexpr (!kByRow) {
      if (a.q_weight) {
        float by[kUnroll];
        row_norms<kDim>(x, a.eps, by);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) scale_row(x[u], by[u], wq);
      }
      if (mine.turned) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) rotation.apply(x[u]);
      }
      uint16_t* out = a.q_out + n_now * a.q_out_stride + (h_now + sub) * kDim;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (h_now + u * kRows + sub < h_end) mine.store(out + u * kRows * kDim, pack_row<kHalf>(x[u]));
    } else {
      const int slot = __ldg(a.slots + n_now);
      const bool write_kv = slot >= 0 && slot < a.total_slots;
      const int page = write_kv ? a.page.quotient(slot) : 0;
      const int64_t row = page * a.page_stride + (write_kv ? slot - page * a.page_size : 0) * a.token_stride;
      float by[kUnroll], top[kUnroll];
      if (a.q_weight || a.k_weight) row_norms<kDim>(x, a.eps, by);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int at = h_now + u * kRows + sub;
        if (at < nq ? a.q_weight != nullptr : at < nq + nk && a.k_weight) scale_row(x[u], by[u], at < nq ? wq : wk);
        if (mine.turned && at < nq + nk) rotation.apply(x[u]);
        top[u] = row_top<true>(x[u], 0.f);
      }
#pragma unroll
      for (int d = kLanes / 2; d > 0; d >>= 1) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], d));
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int at = h_now + u * kRows + sub;
        if (at >= h_end) continue;
        if (at < nq) {
          mine.store(a.q_out + n_now * a.q_out_stride + at * kDim, pack_row<kHalf>(x[u]));
        } else if (write_kv) {
          const bool is_v = at >= nq + nk;
          const int kh = is_v ? at - nq - nk : at - nq;
          const float scale = scale_for(top[u]);
          mine.store_codes((is_v ? a.v_cache : a.k_cache) + row + kh * a.head_stride, quantise_row(x[u], scale));
          if (c == 0) (is_v ? a.v_scale : a.k_scale)[(int64_t)slot * nk + kh] = scale;
        }
      }
    }
  }
  if (!runs_on) return;
  if (a.k_weight) wk = unpack_row<kHalf>(mine.load(a.k_weight));

  // ---- keys and values: run by run, each key head's keys and values for a team
  const int teams = kWarps / team, my_team = warp / team, rank = warp % team;
  const int r0 = rank * kRows + sub;  // this lane's first row of a run; the next is team * kRows behind
  int round = 0;
  for (uint32_t left = leaders; left; left &= left - 1) {
    const int first = __ffs(left) - 1, n = n0 + first;  // its first token
    const int block = __shfl_sync(0xffffffffu, here.block, first);
    // The run: the tokens from n on that lie in this block, as many as it has places.
    const uint32_t other = ~__ballot_sync(0xffffffffu, here.block == block) >> first;
    const int inside = other ? min(__ffs(other) - 1, 32 - first) : 32 - first;
    const int run = min(a.block_tokens, n + inside == n_end ? inside + tail : inside);
    const bool tailed = run > inside;
    uint64_t bit = 0;
    if (lane >= first && lane < first + inside && lane - first < run) bit = 1ull << here.place;
    if (tailed && lane < run - inside) bit |= 1ull << behind[0].place;
    if (tailed && 32 + lane < run - inside) bit |= 1ull << behind[1].place;
    // Tokens of the block that the run writes.
    const uint64_t written = (uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(bit >> 32)) << 32 | __reduce_or_sync(0xffffffffu, (uint32_t)bit);
    const int page = block / a.blocks, b = block - page * a.blocks, slot0 = page * a.page_size + b * a.block_tokens;
    const int64_t block_at = page * a.page_stride + (int64_t)b * a.block_tokens * a.token_stride;
    // Where this lane's rows go.
    int64_t to[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int r = r0 + s * team * kRows;
      to[s] = r < run ? block_at + (__ldg(a.slots + n + r) - slot0) * a.token_stride : 0;
    }
    auto load = [&](int part, uint4 (&in)[kSteps]) {
      const int head = part >> 1;
      const uint16_t* src = (part & 1 ? a.v + (n + r0) * a.v_stride : a.k + (n + r0) * a.k_stride) + head * kDim;
      const int64_t stride = (part & 1 ? a.v_stride : a.k_stride) * (team * kRows);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) in[s] = part < 2 * nk && r0 + s * team * kRows < run ? mine.load(src + s * stride) : none;
    };
    uint4 ahead[kSteps];
    load(slice * teams + my_team, ahead);
    for (int at = slice * teams; at < 2 * nk; at += slices * teams, ++round) {  // the same in the whole CTA
      const int part = at + my_team, head = part >> 1;
      const bool work = part < 2 * nk, is_v = part & 1;
      Row x[kSteps];
      float top = 0.f, old = 0.f;
      float* scale_at = (is_v ? a.v_scale : a.k_scale) + (int64_t)block * nk + head;
      if (work) old = *scale_at;  // in every warp of the team before the exchange below, and so before it changes
#pragma unroll
      for (int s = 0; s < kSteps; ++s) x[s] = unpack_row<kHalf>(ahead[s]);
      load(part + slices * teams, ahead);
      if (work) {
        if (!is_v) {
          if (a.k_weight) {
            float by[kSteps];
            row_norms<kDim>(x, a.eps, by);
#pragma unroll
            for (int s = 0; s < kSteps; ++s) scale_row(x[s], by[s], wk);
          }
          if (mine.turned) {
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
              const float* cs = turns + 2 * (first + min(r0 + s * team * kRows, run - 1)) * pairs + mine.pair;
              Turn<kInterleaved>(cs, cs + pairs).apply(x[s]);
            }
          }
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {
            if (r0 + s * team * kRows >= run) x[s] = Row{};  // no row
          }
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) top = row_top<false>(x[s], top);
        if (__any_sync(0xffffffffu, top == INFINITY)) {
          top = 0.f;
#pragma unroll
          for (int s = 0; s < kSteps; ++s) top = row_top<true>(x[s], top);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      }
      if (team > 1) {
        if (lane == 0) tops[round & 1][warp] = top;
        __syncthreads();  // once a round: the other buffer is read before anyone writes it again
        for (int k = 0; k < team; ++k) top = fmaxf(top, tops[round & 1][my_team * team + k]);
      }
      if (!work) continue;
      const bool begun = !(written & 1) && scale_ok(old);
      const float scale = begun && top <= old * 448.f ? old : scale_for(top);
      uint8_t* rows = (is_v ? a.v_cache : a.k_cache) + head * a.head_stride;
      if (begun && scale != old) {
        // What the block holds already, to the new scale.
        const int tokens = min(a.block_tokens, a.page_size - b * a.block_tokens);
        for (int t = r0; t < tokens; t += team * kRows) {
          if (written >> t & 1) continue;
          uint8_t* p = rows + block_at + t * a.token_stride;
          float held[8];
          unpack_codes8(mine.load_codes(p), held);
          Row r;
#pragma unroll
          for (int j = 0; j < 4; ++j) r.v[j] = pair(held[2 * j] * old, held[2 * j + 1] * old);
          mine.store_codes(p, quantise_row(r, scale));
        }
      }
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        if (r0 + s * team * kRows < run) mine.store_codes(rows + to[s], quantise_row(x[s], scale));
      if (rank == 0 && lane == 0 && scale != old) *scale_at = scale;
    }
  }
}

// Rows read back: eight codes a thread and step, of keys and of values, so that a
// warp's stores lie next to each other.  A CTA takes cta_rows rows at a time; their
// pieces are numbered together.  65,521 rows of 4 x 256 columns: 64 us (6.3 TB/s,
// 0.94 of the copy rate; sixteen codes a thread 78, two steps together 77).
template <bool kHalf>
__global__ void __launch_bounds__(256) draft8_read_kernel(const __grid_constant__ Draft8ReadArgs a) {
  constexpr int kTogether = 4;
  await_grid();
  const int per_head = a.head_dim / 8;  // 8, 16 or 32
  const int head_log2 = a.head_dim == 64 ? 3 : a.head_dim == 128 ? 4 : 5;
  uint32_t bad = 0;
  for (int64_t n0 = (int64_t)blockIdx.x * a.cta_rows; n0 < a.n_rows; n0 += (int64_t)gridDim.x * a.cta_rows) {
    const int pieces = min(a.cta_rows, (int)(a.n_rows - n0)) * a.row_pieces;
    for (int at = threadIdx.x; at < pieces; at += 256 * kTogether) {
      uint2 code[kTogether][2];
      float scale[kTogether][2];
      int64_t row[kTogether];
      int to[kTogether];
#pragma unroll
      for (int u = 0; u < kTogether; ++u) {
        const int i = at + 256 * u;
        row[u] = -1;
        if (i >= pieces) continue;
        const int n = a.piece.quotient(i), piece = i - n * a.row_pieces;
        const int slot = __ldg(a.slots + n0 + n);
        if (slot < 0 || slot >= a.total_slots) {
          if (slot != -1) bad |= DDTREE_ST_BAD_INDEX;
          continue;
        }
        const int head = piece >> head_log2, col = (piece & (per_head - 1)) * 8;
        const int page = a.page.quotient(slot), token = slot - page * a.page_size;
        const int64_t from = page * a.page_stride + token * a.token_stride + head * a.head_stride + col;
        const int64_t s = ((int64_t)page * a.blocks + a.block.quotient(token)) * a.n_kv_heads + head;
        row[u] = n0 + n;
        to[u] = head * a.head_dim + col;
        if (a.k_out) {
          code[u][0] = *reinterpret_cast<const uint2*>(a.k_cache + from);
          scale[u][0] = a.k_scale[s];
        }
        if (a.v_out) {
          code[u][1] = *reinterpret_cast<const uint2*>(a.v_cache + from);
          scale[u][1] = a.v_scale[s];
        }
      }
#pragma unroll
      for (int u = 0; u < kTogether; ++u) {
        if (row[u] < 0) continue;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          uint16_t* out = w ? a.v_out : a.k_out;
          if (!out) continue;
          const bool ok = scale_ok(scale[u][w]);
          if (!ok) bad |= DDTREE_ST_BAD_SCALE;
          float x[8];
          unpack_codes8(code[u][w], x);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = ok ? x[j] * scale[u][w] : 0.f;
          *reinterpret_cast<uint4*>(out + row[u] * (w ? a.v_out_stride : a.k_out_stride) + to[u]) = pack8<kHalf>(x);
        }
      }
    }
  }
  if (bad && a.status) atomicOr(a.status, bad);
}

template <bool kHalf, int kDim>
cudaError_t launch(const Draft8AppendArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int kRows = 256 / kDim;
  const bool by_row = a.block_tokens == 1;
  const int elements = a.block_tokens * kDim, team = elements <= 1024 ? 1 : elements <= 2048 ? 2 : 4;
  // One wave of CTAs where tokens are few: chunks of fewer than eight tokens, down to
  // one, then slices of its heads, in which rows and runs go side by side.
  const int64_t slots = (int64_t)num_sms * 4;
  int chunk = 8;
  while (chunk > 1 && (a.n_tokens + chunk / 2 - 1) / (chunk / 2) <= slots) chunk /= 2;
  const int64_t chunks = (a.n_tokens + chunk - 1) / chunk;
  const int steps = (a.n_heads + (by_row ? 2 * a.n_kv_heads : 0) + kRows - 1) / kRows;
  const int rows_most = (steps + kWarps - 1) / kWarps, runs_most = by_row ? 0 : (2 * a.n_kv_heads * team + kWarps - 1) / kWarps;
  const int slices = (int)std::max<int64_t>(1, std::min<int64_t>(rows_most + runs_most, slots / chunks));
  const int row_slices = by_row || slices == 1 ? slices : a.n_heads == 0 ? 0 : std::max(1, std::min(slices - 1, slices * rows_most / (rows_most + runs_most)));
  // Cosines and sines of a chunk's tokens, and of a block's behind it.
  const size_t smem = (size_t)(chunk + a.block_tokens - 1) * a.rope.rot_dim * sizeof(float);
  static_assert((8 + DDTREE_DRAFT8_MAX_BLOCK / kDim - 1) * (size_t)kDim * sizeof(float) + 64 <= 48 * 1024, "shared memory");
  auto* kernel = a.rope.interleaved ? (by_row ? draft8_append_kernel<kHalf, kDim, true, true> : draft8_append_kernel<kHalf, kDim, true, false>)
                                    : (by_row ? draft8_append_kernel<kHalf, kDim, false, true> : draft8_append_kernel<kHalf, kDim, false, false>);
  return launch_early(kernel, dim3((unsigned)chunks, slices), kThreads, smem, stream, a, chunk, team, row_slices);
}

}  // namespace

cudaError_t launch_draft8_append(const Draft8AppendArgs& a, int num_sms, cudaStream_t stream) {
  if (a.dtype == DDTREE_FP16) {
    return a.head_dim == 64    ? launch<true, 64>(a, num_sms, stream)
           : a.head_dim == 128 ? launch<true, 128>(a, num_sms, stream)
                               : launch<true, 256>(a, num_sms, stream);
  }
  return a.head_dim == 64    ? launch<false, 64>(a, num_sms, stream)
         : a.head_dim == 128 ? launch<false, 128>(a, num_sms, stream)
                             : launch<false, 256>(a, num_sms, stream);
}

cudaError_t launch_draft8_read(const Draft8ReadArgs& args, int num_sms, cudaStream_t stream) {
  Draft8ReadArgs a = args;
  a.cta_rows = std::max(1, 1024 / a.row_pieces);
  a.piece = make_divider(a.row_pieces);
  const int64_t blocks = ((int64_t)a.n_rows + a.cta_rows - 1) / a.cta_rows;
  const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)num_sms * 8);
  return launch_early(a.dtype == DDTREE_FP16 ? draft8_read_kernel<true> : draft8_read_kernel<false>, grid, 256, 0, stream, a);
}

}  // namespace ddtree
