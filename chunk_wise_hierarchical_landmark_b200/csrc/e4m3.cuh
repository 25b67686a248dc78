// The 8-bit cache format: e4m3 codes (sign, 4 exponent bits, 3 mantissa bits;
// largest value 448, no infinities) with one power-of-two scale per block of
// 64 tokens of a KV head.  value = code * scale, exact in fp32 (and in bf16 for
// scales from 2^-124 on; below, the smallest codes' values are under its least
// subnormal): a power of two only moves the exponent, so the one rounding is the
// code's.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace hils {

// The exponent k of the block scale 2^k: the smallest k >= -126 with
// amax <= 448 * 2^k (448 = 1.75 * 2^8), from the bits of a finite amax >= 0.
__device__ __forceinline__ int block_scale_exp(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23);  // biased exponent of amax = 1.m * 2^(e - 127)
  const int k = e - 135 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return k < -126 ? -126 : k;
}
__device__ __forceinline__ float pow2f(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }

// two codes (low byte: a): round to nearest even, values past 448 (infinities
// too) saturate, NaN stays NaN
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// four codes -> two pairs of fp16 values (exact: e4m3's range and precision
// lie inside fp16's)
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 a, z;\n\t"
      "mov.b32 {a, z}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, z;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ float4 e4m3x4_to_f32(uint32_t w) {
  uint32_t lo, hi;
  e4m3x4_to_f16x2(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
  const float2 z = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
  return make_float4(a.x, a.y, z.x, z.y);
}

}  // namespace hils
