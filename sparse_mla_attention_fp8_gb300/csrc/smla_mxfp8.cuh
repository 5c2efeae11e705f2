// MXFP8: e4m3 codes [rows, K] with a scale 2^E per 32 values of a row, kept as
// the byte E + 127.  E is the smallest from -100 up with amax <= 448 * 2^E over
// the group's finite values (as for a block of the paged K/V cache), so that
// dividing by the scale is exact and the only rounding is that to e4m3.
// Infinities saturate; a NaN is stored as e4m3's NaN and spreads to what reads it.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

namespace smla {

constexpr int kMxGroup = 32;

__device__ __forceinline__ uint32_t mx_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// |x| as bits, which are ordered as the values are; 0 for infinities and NaN.
__device__ __forceinline__ uint32_t mx_finite_bits(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}
// E from the bits of amax = (1 + f) 2^e: 448 = 1.75 * 2^8, and the sum carries into
// the exponent where f is above .75.  (Subnormal ones are far below the floor.)
__device__ __forceinline__ int mx_exponent(uint32_t amax_bits) {
  return max(-100, (int)((amax_bits + 0x1fffffu) >> 23) - 127 - 8);
}
__device__ __forceinline__ float mx_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

}  // namespace smla
