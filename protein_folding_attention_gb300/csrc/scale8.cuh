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

// Maxima of magnitudes.  A NaN is skipped (the other operand is taken).
__device__ __forceinline__ float max_abs3(float a, float b, float c) { return fmaxf(fmaxf(fabsf(a), fabsf(b)), c); }
__device__ __forceinline__ float max_abs8(const float (&f)[8]) {
  return max_abs3(f[0], f[1], max_abs3(f[2], f[3], max_abs3(f[4], f[5], max_abs3(f[6], f[7], 0.f))));
}
__device__ __forceinline__ float max_abs(const float (&f)[8]) { return max_abs8(f); }
__device__ __forceinline__ float max_abs(const float (&f)[4]) { return max_abs3(f[0], f[1], max_abs3(f[2], f[3], 0.f)); }
// Where a maximum turns out infinite, infinities become NaN and the maximum is
// taken again: NaN converts to the NaN code, infinity would convert to 448.
__device__ __forceinline__ float infinity_to_nan(float x) { return fabsf(x) > FLT_MAX ? __int_as_float(0x7FFFFFFF) : x; }

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
// Codes of elements (none infinite) times the inverse scale, the first in the low
// byte.  The product with a power of two is exact.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi, float inverse) {
  uint16_t r;
  uint64_t in, two, by;
  asm("mov.b64 %0, {%1, %2};" : "=l"(in) : "f"(lo), "f"(hi));
  asm("mov.b64 %0, {%1, %1};" : "=l"(by) : "f"(inverse));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(two) : "l"(in), "l"(by));
  asm("{\n .reg .f32 a, b;\n mov.b64 {a, b}, %1;\n cvt.rn.satfinite.e4m3x2.f32 %0, b, a;\n}\n" : "=h"(r) : "l"(two));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_four(float a, float b, float c, float d, float inverse) {
  return e4m3_pair(a, b, inverse) | e4m3_pair(c, d, inverse) << 16;
}

}  // namespace evo
