// Launcher of the 8-bit matrix product with block scales.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "layout.cuh"

namespace evo {

// Rows of e4m3 codes with a scale per 128 of them; `shift` 7 where 128 rows
// share a scale.
struct Operand8 {
  const void* codes;
  int64_t ld;             // bytes
  const uint8_t* scales;
  int64_t s_row, s_group;
  int shift;
};

struct Matmul8Call {
  Operand8 a, b;          // [M, K], [N, K]
  int M, N, K;
  void* out;              // [M, N], row stride ld_out (elements)
  int64_t ld_out;
  const void* add;        // likewise, or NULL
  int64_t ld_add;
  bool f32;               // type of out and add
  float* ws;
  WaitCfg wait;
};

// How a product is cut up: tiles of 128 rows of one operand by bq rows of the
// other; the sum over K in `splits` pieces of per_split groups.
struct Matmul8Plan {
  bool staged;            // a's rows are the 128, else b's
  int bq, tiles_p, tiles_q, groups, per_split, splits;
};
Matmul8Plan matmul8_plan(int M, int N, int K, int sms);
size_t matmul8_workspace_bytes(int M, int N, int K, int sms);

cudaError_t matmul8(const Matmul8Call& c, const Matmul8Plan& plan, int sms, cudaStream_t st, bool* tmap_ok);

}  // namespace evo
