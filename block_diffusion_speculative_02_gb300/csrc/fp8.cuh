// Values in 8-bit floating point (e4m3) with a scale for each block of 128: what the calls
// of fp8_rows.cu and fp8_linear.cu share.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "host.h"

namespace dflash {
namespace fp8 {

constexpr int kBlockK = 128;      // columns (and, of weights, rows) that share a scale
constexpr float kMax = 448.f;     // the largest e4m3 value

inline long long blocks(long long n) { return (n + kBlockK - 1) / kBlockK; }

// The largest magnitude that a scale is made of is at least 2^-117: the scale is then at
// least 2^-126 and its reciprocal finite.
__device__ __forceinline__ float floor_of_max() { return __uint_as_float((127 - 117) << 23); }

// Bits of |x|: they compare as the magnitudes do, infinities and NaN above all.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// scale = a / 448 and what the values are multiplied by, 448 / a, for the block's largest
// magnitude (its bits).  A block with an infinity or NaN gets a scale and codes of NaN, so
// that it shows in whatever is made of it.
__device__ __forceinline__ void scale_of(uint32_t max_bits, float* scale, float* inverse) {
  float a = fmaxf(__uint_as_float(max_bits), floor_of_max());
  if (max_bits >= 0x7F800000u) a = __uint_as_float(0x7FC00000u);
  *scale = a / kMax;
  *inverse = kMax / a;
}

// 16 values times r as e4m3 codes (to nearest, ties to even, saturating; NaN stays NaN).
__device__ __forceinline__ uint4 codes16(const float (&v)[16], float r) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i] * r, v[4 * i + 1] * r),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2] * r, v[4 * i + 3] * r),
                                                 __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | hi << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 bf16 values (32 bytes, 16-byte aligned) as fp32.
__device__ __forceinline__ void widen16(const uint4 (&x)[2], float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
      v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ void load16(const uint16_t* p, uint4 (&x)[2]) {
  x[0] = reinterpret_cast<const uint4*>(p)[0];
  x[1] = reinterpret_cast<const uint4*>(p)[1];
}

// The largest magnitude (as bits) of the 8 consecutive lanes that hold a block of 128.
__device__ __forceinline__ uint32_t max8(uint32_t m) {
#pragma unroll
  for (int o = 4; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

__device__ __forceinline__ uint32_t max16(const float (&v)[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, abs_bits(v[i]));
  return m;
}

}  // namespace fp8
}  // namespace dflash
