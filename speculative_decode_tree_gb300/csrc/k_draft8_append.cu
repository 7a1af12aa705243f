// The drafter's new queries, keys and values with a cache in 8 bits
// (include/ddtree_draft8.h): head norms, rotation, quantisation as the rows are
// written; and rows read back.
//
// Queries go as in the 16-bit append: a warp per token or slice of its heads,
// sines and cosines in registers.  So do keys and values where every token has
// scales of its own (blocks of one token).
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
#include "rope.cuh"

namespace ddtree {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 3;   // head steps of a query whose loads are in flight together
constexpr int kSteps = 4;    // row steps of a warp in a run

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
// x / s for eight numbers: a product where s is a power of two (also exact), else the quotient.
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float s) {
  float y[8];
  if ((__float_as_uint(s) & 0x7fffffu) == 0) {
    const float inv = __uint_as_float((254u << 23) - __float_as_uint(s));
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = x[j] * inv;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = __fdiv_rn(x[j], s);
  }
  return make_uint2(to_codes(y[0], y[1], y[2], y[3]), to_codes(y[4], y[5], y[6], y[7]));
}

// What a lane needs of the rotation: it has the columns 8 c .. 8 c + 7 of every
// row.  Interleaved, those are four pairs of its own; in the half layout eight
// pairs that it shares with the lane of the other half, and each computes four.
template <int kDim, bool kInterleaved>
struct Turner {
  static constexpr int kLanes = kDim / 8, kTurns = kInterleaved ? 4 : 8;
  uint64_t turns[4];
  int other_lane;
  bool turned, first;
  __device__ __forceinline__ Turner(const RopeArgs& rope, int lane) {
    const int c = lane % kLanes, half = rope.rot_dim / 16;
    turned = 8 * c < rope.rot_dim;
    first = c < half;
    const int other = !turned ? c : first ? c + half : c - half;
    other_lane = (lane & ~(kLanes - 1)) + other;
    const int pair = !turned ? 0 : kInterleaved ? 4 * c : first ? 8 * c : 8 * other + 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) turns[j] = rope.turns[pair + j];
  }
  __device__ __forceinline__ void at(int pos, float mscale, float2 (&cs)[kTurns]) const {
    float2 mine[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) mine[j] = turn(turns[j], pos, mscale);
    if constexpr (kInterleaved) {
#pragma unroll
      for (int j = 0; j < 4; ++j) cs[j] = mine[j];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 theirs = make_float2(__shfl_sync(0xffffffffu, mine[j].x, other_lane), __shfl_sync(0xffffffffu, mine[j].y, other_lane));
        // x cos - y sin for a first element, x cos + y sin for a second one, y its partner.
        cs[j] = first ? make_float2(mine[j].x, -mine[j].y) : theirs;
        cs[j + 4] = first ? make_float2(theirs.x, -theirs.y) : mine[j];
      }
    }
  }
  __device__ __forceinline__ void apply(float (&x)[8], const float2 (&cs)[kTurns]) const {
    if constexpr (kInterleaved) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = x[2 * j], o = x[2 * j + 1];
        x[2 * j] = turned ? e * cs[j].x - o * cs[j].y : e;
        x[2 * j + 1] = turned ? e * cs[j].y + o * cs[j].x : o;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float y = __shfl_sync(0xffffffffu, x[j], other_lane);
        if (turned) x[j] = x[j] * cs[j].x + y * cs[j].y;
      }
    }
  }
};

// The norm of a row that kDim / 8 lanes hold.
template <bool kHalf, int kDim>
__device__ __forceinline__ void norm_row(float (&x)[8], const uint4& weight, float eps) {
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
#pragma unroll
  for (int d = kDim / 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  const float scale = rsqrtf(sum * (1.f / kDim) + eps);
  float w[8];
  unpack8<kHalf>(weight, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = x[j] * scale * w[j];
}

// Grid: chunks of `chunk` tokens (a power of two), slices of their heads.
// team: warps of a run.
template <bool kHalf, int kDim, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 4) draft8_append_kernel(const __grid_constant__ Draft8AppendArgs a, int chunk, int team) {
  constexpr int kLanes = kDim / 8;        // lanes of a row
  constexpr int kRows = 32 / kLanes;      // rows of a warp's step
  using Turn = Turner<kDim, kInterleaved>;
  __shared__ float tops[2][kWarps];
  await_grid();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = lane % kLanes, sub = lane / kLanes;
  const int slice = blockIdx.y, slices = gridDim.y;
  const int n0 = blockIdx.x * chunk, n_end = min(n0 + chunk, a.n_tokens);
  const Turn rotation(a.rope, lane);
  const uint4 none = make_uint4(0, 0, 0, 0);
  const uint4 wq = a.q_weight ? __ldg(reinterpret_cast<const uint4*>(a.q_weight) + c) : none;
  const uint4 wk = a.k_weight ? __ldg(reinterpret_cast<const uint4*>(a.k_weight) + c) : none;
  if (slice == 0 && warp == 0 && a.status && n0 + lane < n_end) {
    const int pos = __ldg(a.positions + n0 + lane), slot = __ldg(a.slots + n0 + lane);
    if (pos < -1) atomicOr(a.status, DDTREE_ST_BAD_LENGTH);
    else if (pos >= 0 && (slot < -1 || slot >= a.total_slots)) atomicOr(a.status, DDTREE_ST_BAD_INDEX);
  }

  // ---- rows on their own: queries, and where every token has its own scale keys and values too
  const bool by_row = a.block_tokens == 1;
  const int nq = a.n_heads, nk = a.n_kv_heads, row_heads = by_row ? nq + 2 * nk : nq;
  {
    const int per_token = chunk < kWarps ? kWarps / chunk : 1;  // warps of a token
    const int steps = (row_heads + kRows - 1) / kRows, parts = slices * per_token;
    const int part = slice * per_token + warp % per_token, part_steps = (steps + parts - 1) / parts;
    const int h_begin = part * part_steps * kRows, h_end = min(h_begin + part_steps * kRows, row_heads);
    for (int n = n0 + warp / per_token; n < n_end && h_begin < h_end; n += kWarps / per_token) {
      const int pos = __ldg(a.positions + n), slot = __ldg(a.slots + n);
      const uint16_t *q = a.q + n * a.q_stride, *k = a.k + n * a.k_stride, *v = a.v + n * a.v_stride;
      uint16_t* out = a.q_out + n * a.q_out_stride;
      const bool write_kv = slot >= 0 && slot < a.total_slots;
      const int page = write_kv ? a.page.quotient(slot) : 0;
      const int64_t row = page * a.page_stride + (write_kv ? slot - page * a.page_size : 0) * a.token_stride;
      float2 cs[Turn::kTurns];
      for (int base = h_begin; base < h_end; base += kRows * kUnroll) {
        uint4 in[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int h = base + u * kRows + sub;
          const uint16_t* src = h < nq ? q + h * kDim : h < nq + nk ? k + (h - nq) * kDim : v + (h - nq - nk) * kDim;
          in[u] = h < h_end ? reinterpret_cast<const uint4*>(src)[c] : none;  // plain loads: q_out may be q
        }
        if (pos < 0) break;
        if (base == h_begin) rotation.at(pos, a.rope.mscale, cs);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          if (base + u * kRows >= h_end) break;  // the same in the whole warp
          const int h = base + u * kRows + sub;
          const bool is_q = h < nq, is_v = h >= nq + nk;
          float x[8];
          unpack8<kHalf>(in[u], x);
          if (a.q_weight || a.k_weight) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = x[j];
            norm_row<kHalf, kDim>(y, is_q ? wq : wk, a.eps);
            if (!is_v && (is_q ? a.q_weight : a.k_weight)) {
#pragma unroll
              for (int j = 0; j < 8; ++j) x[j] = y[j];
            }
          }
          float y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = x[j];
          rotation.apply(y, cs);
          if (!is_v) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = y[j];
          }
          if (by_row) {
            float top = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float m = fabsf(x[j]);
              if (m < INFINITY) top = fmaxf(top, m);
            }
#pragma unroll
            for (int d = kLanes / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            if (!is_q && h < h_end && write_kv) {
              const float scale = scale_for(top);
              const int kh = is_v ? h - nq - nk : h - nq;
              *reinterpret_cast<uint2*>((is_v ? a.v_cache : a.k_cache) + row + kh * a.head_stride + 8 * c) = quantise8(x, scale);
              if (c == 0) (is_v ? a.v_scale : a.k_scale)[(int64_t)slot * nk + kh] = scale;
            }
          }
          if (is_q && h < h_end) reinterpret_cast<uint4*>(out + h * kDim)[c] = pack8<kHalf>(x);
        }
      }
    }
  }
  if (by_row) return;

  // ---- keys and values: the chunk's runs, each key head's keys and values an item
  auto block_of = [&](int n) {  // number of the token's block, -1 where nothing is written
    if (n < 0 || n >= a.n_tokens) return -1;
    const int pos = __ldg(a.positions + n), slot = __ldg(a.slots + n);
    if (pos < 0 || slot < 0 || slot >= a.total_slots) return -1;
    const int page = a.page.quotient(slot);
    return page * a.blocks + a.block.quotient(slot - page * a.page_size);
  };
  const int mine = n0 + lane < n_end ? block_of(n0 + lane) : -1;
  int before = __shfl_up_sync(0xffffffffu, mine, 1);
  if (lane == 0) before = block_of(n0 - 1);
  const uint32_t leaders = __ballot_sync(0xffffffffu, mine >= 0 && mine != before);
  const int teams = kWarps / team, my_team = warp / team, rank = warp % team;
  const uint32_t per_run = 2 * nk, items = __popc(leaders) * per_run;
  int round = 0;
  for (uint32_t at = slice * teams; at < items; at += slices * teams, ++round) {  // the same in the whole CTA
    const uint32_t item = at + my_team;
    const bool work = item < items;
    float x[kSteps][8], top = 0.f, old = 0.f;
    int n = 0, block = 0, run = 0, head = 0;
    bool is_v = false;
    uint64_t written = 0;  // tokens of the block that the run writes
    float* scale_at = nullptr;
    if (work) {
      const uint32_t which = item / per_run, part = item - which * per_run;
      head = part >> 1;
      is_v = part & 1;
      uint32_t left = leaders;
      for (uint32_t k = 0; k < which; ++k) left &= left - 1;
      const int first = __ffs(left) - 1;
      n = n0 + first;
      block = __shfl_sync(0xffffffffu, mine, first);
      scale_at = (is_v ? a.v_scale : a.k_scale) + (int64_t)block * nk + head;
      old = *scale_at;  // in every warp of the team before the exchange below, and so before it changes
      // The run: the tokens from n on that lie in this block, as many as it has places.
      uint32_t same[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        same[k] = __ballot_sync(0xffffffffu, 32 * k + lane < a.block_tokens && block_of(n + 32 * k + lane) == block);
      run = ~same[0] ? __ffs(~same[0]) - 1 : ~same[1] ? 31 + __ffs(~same[1]) : 64;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t lo = 0, hi = 0;
        if (32 * k + lane < run) {
          const int slot = __ldg(a.slots + n + 32 * k + lane), in_page = slot - a.page.quotient(slot) * a.page_size;
          const int t = in_page - a.block.quotient(in_page) * a.block_tokens;
          (t < 32 ? lo : hi) = 1u << (t & 31);
        }
        written |= (uint64_t)__reduce_or_sync(0xffffffffu, hi) << 32 | __reduce_or_sync(0xffffffffu, lo);
      }
      const uint16_t* src = is_v ? a.v + head * kDim : a.k + head * kDim;
      const int64_t stride = is_v ? a.v_stride : a.k_stride;
      uint4 in[kSteps];
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int r = (s * team + rank) * kRows + sub;
        in[s] = r < run ? __ldg(reinterpret_cast<const uint4*>(src + (n + r) * stride) + c) : none;
      }
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int r0 = (s * team + rank) * kRows;
        unpack8<kHalf>(in[s], x[s]);
        if (!is_v && r0 < run) {  // the same in the whole warp
          if (a.k_weight) norm_row<kHalf, kDim>(x[s], wk, a.eps);
          float2 cs[Turn::kTurns];
          rotation.at(__ldg(a.positions + n + min(r0 + sub, run - 1)), a.rope.mscale, cs);
          rotation.apply(x[s], cs);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float m = fabsf(x[s][j]);
          if (m < INFINITY) top = fmaxf(top, m);
        }
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
    const int page = block / a.blocks, b = block - page * a.blocks;
    uint8_t* rows = (is_v ? a.v_cache : a.k_cache) + page * a.page_stride + (int64_t)b * a.block_tokens * a.token_stride +
                    head * a.head_stride + 8 * c;
    if (begun && scale != old) {
      // What the block holds already, to the new scale.
      const int tokens = min(a.block_tokens, a.page_size - b * a.block_tokens);
      for (int t = rank * kRows + sub; t < tokens; t += team * kRows) {
        if (written >> t & 1) continue;
        uint2* p = reinterpret_cast<uint2*>(rows + t * a.token_stride);
        float held[8];
        unpack_codes8(*p, held);
#pragma unroll
        for (int j = 0; j < 8; ++j) held[j] *= old;
        *p = quantise8(held, scale);
      }
    }
    const int slot0 = page * a.page_size + b * a.block_tokens;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int r = (s * team + rank) * kRows + sub;
      if (r < run) *reinterpret_cast<uint2*>(rows + (__ldg(a.slots + n + r) - slot0) * a.token_stride) = quantise8(x[s], scale);
    }
    if (rank == 0 && lane == 0 && scale != old) *scale_at = scale;
  }
}

// Rows read back: eight codes a thread and step, of keys and of values.
template <bool kHalf>
__global__ void __launch_bounds__(256) draft8_read_kernel(const __grid_constant__ Draft8ReadArgs a) {
  constexpr int kTogether = 4;
  await_grid();
  const int64_t pieces = (int64_t)a.n_rows * a.row_pieces, stride = (int64_t)gridDim.x * 256;
  const int per_head = a.head_dim / 8;
  uint32_t bad = 0;
  for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < pieces; at += stride * kTogether) {
    uint2 code[kTogether][2];
    float scale[kTogether][2];
    int64_t to[kTogether];
    int row[kTogether];
#pragma unroll
    for (int u = 0; u < kTogether; ++u) {
      const int64_t i = at + u * stride;
      row[u] = -1;
      if (i >= pieces) continue;
      const int n = (int)(i / a.row_pieces), piece = (int)(i - (int64_t)n * a.row_pieces);
      const int slot = __ldg(a.slots + n);
      if (slot < 0 || slot >= a.total_slots) {
        if (slot != -1) bad |= DDTREE_ST_BAD_INDEX;
        continue;
      }
      const int head = piece / per_head, col = (piece - head * per_head) * 8;
      const int page = a.page.quotient(slot), token = slot - page * a.page_size;
      const int64_t from = page * a.page_stride + token * a.token_stride + head * a.head_stride + col;
      const int64_t s = ((int64_t)page * a.blocks + a.block.quotient(token)) * a.n_kv_heads + head;
      row[u] = n;
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
        float x[8];
        unpack_codes8(code[u][w], x);
        const bool ok = scale_ok(scale[u][w]);
        if (!ok) bad |= DDTREE_ST_BAD_SCALE;
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = ok ? x[j] * scale[u][w] : 0.f;
        *reinterpret_cast<uint4*>(out + row[u] * (w ? a.v_out_stride : a.k_out_stride) + to[u]) = pack8<kHalf>(x);
      }
    }
  }
  if (bad && a.status) atomicOr(a.status, bad);
}

template <bool kHalf, int kDim>
cudaError_t launch(const Draft8AppendArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int kRows = 256 / kDim;
  const int elements = a.block_tokens * kDim, team = elements <= 1024 ? 1 : elements <= 2048 ? 2 : 4;
  // Chunks of up to 32 tokens; fewer tokens take smaller chunks and slices of
  // the heads, until there are some CTAs for each SM.
  const int items = a.block_tokens == 1 ? 0 : 2 * a.n_kv_heads * team;  // warps of a run
  const int steps = (a.n_heads + (a.block_tokens == 1 ? 2 * a.n_kv_heads : 0) + kRows - 1) / kRows;
  const int most = std::max(1, std::max((items + kWarps - 1) / kWarps, steps / kWarps));
  int chunk = 32;
  while (chunk > 1 && (int64_t)((a.n_tokens + chunk - 1) / chunk) * most < num_sms * 4) chunk /= 2;
  const int64_t chunks = (a.n_tokens + chunk - 1) / chunk;
  const int slices = (int)std::max<int64_t>(1, std::min<int64_t>(most, (num_sms * 4 + chunks - 1) / chunks));
  return launch_early(a.rope.interleaved ? draft8_append_kernel<kHalf, kDim, true> : draft8_append_kernel<kHalf, kDim, false>,
                      dim3((unsigned)chunks, slices), kThreads, 0, stream, a, chunk, team);
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

cudaError_t launch_draft8_read(const Draft8ReadArgs& a, int num_sms, cudaStream_t stream) {
  const int64_t blocks = ((int64_t)a.n_rows * a.row_pieces + 255) / 256;
  const unsigned grid = (unsigned)std::min<int64_t>(blocks, (int64_t)num_sms * 8);
  return launch_early(a.dtype == DDTREE_FP16 ? draft8_read_kernel<true> : draft8_read_kernel<false>, grid, 256, 0, stream, a);
}

}  // namespace ddtree
