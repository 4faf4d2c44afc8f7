// The 8-bit KV cache format, shared by the kernels that write, read back and
// attend over it.
//
// A cached row (one token, one KV head, d values) is d e4m3 codes and one scale
// byte e standing for the factor 2^(e - 127); the row's values are code * 2^(e - 127).
// A power of two keeps every step exact except the rounding to e4m3 itself: the
// division by the scale, the code times the scale, and the scale's use as a
// factor of a score.  e4m3 is a floating-point format, so a free scale would buy
// no mantissa bits, only up to one binade at the bottom of the range.  No bf16 row needs
// a byte above 247 (448 * 2^120 passes bf16's largest value); larger ones, which a cache
// filled by other means may hold, count as 247.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace attn {
namespace q8 {

constexpr int kMaxScaleByte = 247;

// Scale byte of a row with largest magnitude amax (finite, >= 0): the smallest
// e >= 1 with amax <= 448 * 2^(e - 127).  448 = 1.75 * 2^8, so with amax =
// 1.f * 2^(E - 127) that is E - 8, or E - 7 when 1.f > 1.75.
__device__ __forceinline__ int scale_byte(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = (int)(bits >> 23) - ((bits & 0x7fffffu) > 0x600000u ? 7 : 8);
  return max(e, 1);
}

// 2^(e - 127) for a scale byte, and its reciprocal for bytes from scale_byte()
// (1..247: both are normal numbers).
__device__ __forceinline__ float scale_of(int e) {
  return __uint_as_float(e == 0 ? 0x00400000u : (uint32_t)e << 23);
}
__device__ __forceinline__ float inv_scale_of(int e) {
  return __uint_as_float((uint32_t)(254 - e) << 23);
}

// Two fp32 values as e4m3 codes (round to nearest even, saturating at 448): lo in the low byte.
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four codes of a 32-bit word as two f16 pairs (exact: e4m3 values are f16 values):
// lo = (byte 0, byte 1), hi = (byte 2, byte 3).
__device__ __forceinline__ void codes4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

}  // namespace q8
}  // namespace attn
