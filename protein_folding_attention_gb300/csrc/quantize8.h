// Launcher of the quantisation to e4m3 with power-of-two scales.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace evo {

struct Quantize8Call {
  const void* x;         // [R, K], row stride ld (elements)
  int64_t R, K, ld;
  bool blocks;           // one scale per 128 x 128 block, held once (scales)
  uint8_t* codes;        // [R, K], row stride ldc, or NULL
  int64_t ldc;
  uint8_t* scales;       // by row (blocks: by 128 rows) and group of columns
  int64_t s_row, s_group;
  uint8_t* codes_t;      // [K, R], row stride ldt, or NULL
  int64_t ldt;
  uint8_t* scales_t;     // by column and group of rows (not with blocks)
  int64_t st_row, st_group;
};

cudaError_t quantize8(const Quantize8Call& c, bool f32, cudaStream_t st);

}  // namespace evo
