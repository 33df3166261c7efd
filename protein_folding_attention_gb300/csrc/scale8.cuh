// e4m3 codes with a power-of-two scale for each group of 128 elements.
//
// The scale is the smallest 2^k with max|x| <= 448 * 2^k (k >= -127; 1 for a
// group of zeros), held as its exponent in 8 bits (k + 127), which is what the
// tensor core multiplies by on its own.  With a power of two x / 2^k is exact, so
// a code is off by the one rounding to e4m3 alone: half a step, 2^-4 of the
// value from 2^-6 on and 2^-10 below, in units of the scale.  Against a scale of
// max|x| / 448 the range in use is up to a factor of two shorter at its lower
// end; the relative error above it is the same.
//
// An infinite or NaN element takes the NaN code and has no part in the maximum.
#pragma once
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

namespace evo {

constexpr int kGroup8 = 128;  // elements that share a scale

// |x| for a group's maximum.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= FLT_MAX ? a : 0.f;
}

// The scale's exponent in 8 bits: from the exponent and mantissa of the
// largest magnitude, 1.m 2^e with 448 = 1.75 * 2^8.
__device__ __forceinline__ uint32_t scale_code(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - ((u & 0x7FFFFFu) > 0x600000u ? 7 : 8);
  return amax > 0.f ? (uint32_t)max(e, 0) : 127u;
}
// 2^-k for the code k + 127 (k from -127 to 120).
__device__ __forceinline__ float scale_inverse(uint32_t code) {
  return code < 254u ? __uint_as_float((254u - code) << 23) : 0.f;
}
// Codes of two elements times the inverse scale, the first in the low byte.
// x * 0 is NaN for an infinite or NaN x and nothing otherwise; without it the
// conversion would turn infinity into 448.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi, float inverse) {
  uint16_t r;
  const float a = fmaf(lo, 0.f, lo * inverse), b = fmaf(hi, 0.f, hi * inverse);
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

}  // namespace evo
