// Launchers of the residual add with dropout, of the norm with 8-bit output,
// and of its gradients.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "block_norm.h"
#include "philox.cuh"

namespace evo {

constexpr int kNorm8MaxCtas = 608;  // CTAs of a backward launch (one partial sum each)

// One call on the row space n[0] x n[1] x n[2] (merged where every operand
// allows it); operands that are not given have p = NULL.
struct Norm8Call {
  int n[3];
  int given[3];     // the row axes before they were merged (the mask's)
  bool turned;      // I and J are exchanged: a row's index is not its mask row's
  int C;
  bool rms;
  float eps;
  bool drop;        // mask is in use
  DropMask mask;
  RowOperand x, u, x1;          // dropout: x, u and out; norm: x, u and x1
  uint8_t* codes;
  int64_t codes_s[3];
  uint8_t* scales;
  int64_t scales_s[3], scales_g;  // by row axis and by group
  const float *gamma, *beta;
  RowOperand dx1, dy, dx, du;   // backward (x1 is read)
  float *dgamma, *dbeta, *ws;
};

size_t norm8_bwd_workspace_bytes(int C);

// (stream type, block type): (bf16, bf16), (fp32, bf16), (fp32, fp32); the
// dropout alone also (bf16, fp32), which the gradient of the second is
cudaError_t dropout_add_bf16(const Norm8Call& c, cudaStream_t st);
cudaError_t dropout_add_narrow(const Norm8Call& c, cudaStream_t st);
cudaError_t dropout_add_mixed(const Norm8Call& c, cudaStream_t st);
cudaError_t dropout_add_f32(const Norm8Call& c, cudaStream_t st);
cudaError_t norm8_fwd_bf16(const Norm8Call& c, cudaStream_t st);
cudaError_t norm8_fwd_mixed(const Norm8Call& c, cudaStream_t st);
cudaError_t norm8_fwd_f32(const Norm8Call& c, cudaStream_t st);
cudaError_t norm8_bwd_bf16(const Norm8Call& c, cudaStream_t st);
cudaError_t norm8_bwd_mixed(const Norm8Call& c, cudaStream_t st);
cudaError_t norm8_bwd_f32(const Norm8Call& c, cudaStream_t st);

}  // namespace evo
