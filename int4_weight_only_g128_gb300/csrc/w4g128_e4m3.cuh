// Conversions of e4m3 codes (1 sign, 4 exponent and 3 mantissa bits; largest
// 448, NaN 0x7F; steps of 2^-9 below 2^-6), two at a time.
#pragma once
#include <cstdint>

namespace w4g128 {

constexpr float kE4M3Max = 448.f;

// Codes of lo (low byte) and hi, to nearest, ties to even; |x| up to 448.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// fp16 holds every e4m3 value.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}

}  // namespace w4g128
