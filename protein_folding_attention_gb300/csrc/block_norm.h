// Launchers of the block norm: the norm after a block, its gate, the residual
// scale and the norm before the next block, and their gradients.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace evo {

// One operand of the block norm on the row space [B, I, J]: base address and
// element strides along the three row axes.  The channels are contiguous.
struct RowOperand {
  void* p;
  int64_t s[3];
};

constexpr int kNormMaxC = 4096;   // channels of a row
constexpr int kNormMaxCtas = 640; // CTAs of a backward launch (one partial sum each)
constexpr int kNormMaxItems = 4 * kNormMaxCtas;  // pieces of shared gate rows (one partial sum each)

struct BlockNormCall {
  int n[3];  // B, I, J
  int C;
  bool rms;
  float eps;
  RowOperand x;     // forward: x; backward: x1
  RowOperand u, gate;
  const float *scale, *gamma_post, *beta_post, *gamma_pre, *beta_pre;
  RowOperand x1, y;           // forward outputs
  RowOperand dx1, dy;         // backward inputs
  RowOperand dx, du, dgate;   // backward outputs
  float *dscale, *dgamma_post, *dbeta_post, *dgamma_pre, *dbeta_pre;
  float* ws;                  // backward workspace
};

// Bytes of the backward's workspace.
size_t block_norm_bwd_workspace_bytes(int C);

// One pair of launchers per (stream type, block type): the residual stream
// (x, x1, dx1, dx) and the block's own tensors (u, gate, y, their gradients).
cudaError_t block_norm_fwd_bf16(const BlockNormCall& c, cudaStream_t st);
cudaError_t block_norm_bwd_bf16(const BlockNormCall& c, cudaStream_t st);
cudaError_t block_norm_fwd_mixed(const BlockNormCall& c, cudaStream_t st);
cudaError_t block_norm_bwd_mixed(const BlockNormCall& c, cudaStream_t st);
cudaError_t block_norm_fwd_f32(const BlockNormCall& c, cudaStream_t st);
cudaError_t block_norm_bwd_f32(const BlockNormCall& c, cudaStream_t st);

}  // namespace evo
