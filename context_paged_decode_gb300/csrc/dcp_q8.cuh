// e4m3 numbers and the scales of 8-bit pages (dcp_q8_cache.cu,
// dcp_scored.cu, dcp_scored_mma.cu).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "dcp_common.cuh"

namespace dcp {

constexpr int kScaleFloats = 4;   // of a page and head: keys', values', two unused

// Four e4m3 numbers (the low byte first) as fp16, which holds them exactly.
__device__ __forceinline__ void e4m3x4_f16(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}

__device__ __forceinline__ float4 e4m3x4_f32(uint32_t four) {
  uint32_t a, b;
  e4m3x4_f16(four, a, b);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  return make_float4(x.x, x.y, y.x, y.y);
}

// Four numbers to e4m3: the nearest, ties to even; beyond +-448, infinities
// among them, +-448; NaN stays NaN.
__device__ __forceinline__ uint32_t f32x4_e4m3(float4 x) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x.x, x.y), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x.z, x.w), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// The smallest power of two s >= 2^-60 with top / s <= 448 = 1.75 * 2^8, by the
// bits of top (finite, >= 0).  Scales are powers of two: dividing by one is
// exact, so a number is rounded once, and a page whose scale grows loses only
// what falls below the smallest numbers of the larger scale.  A power of two
// costs e4m3 nothing but up to one step of its range at the bottom.
__device__ __forceinline__ float scale_for(float top) {
  const int bits = __float_as_int(top);
  int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
  e = max(e, -60);
  return __int_as_float((e + 127) << 23);
}

}  // namespace dcp
