// The position rotation and 16-byte pieces of 16-bit rows, shared by the
// append kernels.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace ddtree {

// (cos, sin) * mscale of position * f, f a 64-bit fraction of a turn.  The
// product modulo 2^64 is the angle modulo one turn; its upper 32 bits, signed,
// are the angle in [-1/2, 1/2) turns.
__device__ __forceinline__ float2 turn(uint64_t f, int32_t position, float mscale) {
  const uint32_t p = (uint32_t)position;
  const uint32_t t = (uint32_t)(f >> 32) * p + __umulhi((uint32_t)f, p);
  float s, c;
  sincospif((float)(int32_t)t * 0x1p-31f, &s, &c);
  return make_float2(c * mscale, s * mscale);
}

template <bool kHalf>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (kHalf) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  } else {
    return make_float2(bf16_lo(v), bf16_hi(v));
  }
}
template <bool kHalf>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if constexpr (kHalf) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <bool kHalf>
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2<kHalf>(w[i]);
    x[2 * i] = p.x;
    x[2 * i + 1] = p.y;
  }
}
template <bool kHalf>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2<kHalf>(x[0], x[1]), pack2<kHalf>(x[2], x[3]), pack2<kHalf>(x[4], x[5]),
                    pack2<kHalf>(x[6], x[7]));
}

}  // namespace ddtree
