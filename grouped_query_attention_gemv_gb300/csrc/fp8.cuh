// Rows of an 8-bit cache: 128 values of one token and KV head as e4m3 times
// 2^e, e the least integer in [LEAST_E, MOST_E] with max |x| <= 448 * 2^e (448 is
// the largest e4m3). Scales that are powers of two cost nothing: a product
// with one is exact, so each value is rounded once, by half a step of 2^-3
// relative at most, and the way back to bf16 is exact (4 significant bits); a
// float format gains nothing from a finer scale. LEAST_E keeps the products of
// the decode attention normal: rows below 2^-91 are held in steps of 2^-109. At
// MOST_E, 248 and more would round to 256, and 256 x 2^120 is past the largest
// float: what is past 240 is held as 240, by 2^-4 of itself off at most as well.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace gqa {

constexpr int LEAST_E = -100, MOST_E = 120;
constexpr float MOST_UNITS = 240.f;  // at MOST_E

// e for the largest |x| of a row, given as its bits (finite).
__device__ __forceinline__ int row_exponent(uint32_t bits) {
  // |x| = 1.m x 2^k; 448 = 1.75 x 2^8
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);
  return min(max(e, LEAST_E), MOST_E);
}
// 2^e, e in [-126, 127]
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// 2^e of a scale byte
__device__ __forceinline__ float scale_value(uint32_t byte) { return __uint_as_float(byte << 23); }

// A value of a row at MOST_E, in units, within reach of what reads it (NaN stays).
__device__ __forceinline__ float within_reach(float x) { return fabsf(x) > MOST_UNITS ? copysignf(MOST_UNITS, x) : x; }
// Two values to e4m3 (ties to even, in range), x in the lower byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float x, float y) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
  return r;
}
// The lower and the upper two e4m3 of a word as f16 pairs (exact).
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi) : "r"(w));
}

}  // namespace gqa
