// Division of indexes by a divisor that a launch knows.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace evo {

// q = r / d for r < 2^31, by the high half of a product.
struct Divide {
  uint32_t d, mul, shift;
};
__device__ __forceinline__ uint32_t quotient(const Divide& v, uint32_t r) {
  return (uint32_t)((uint64_t)r * v.mul >> 31 >> v.shift);
}
inline Divide divide_by(uint32_t d) {
  uint32_t s = 0;
  while (((uint64_t)1 << s) < d) ++s;  // 2^s >= d: r * (2^(31+s) / d + 1) is off by r / 2^(31+s) < 1 / d
  return Divide{d, (uint32_t)(((uint64_t)1 << (31 + s)) / d + 1), s};
}

}  // namespace evo
