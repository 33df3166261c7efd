// The block norm's kernels for: bf16 residual stream, bf16 block tensors.
#include "block_norm.cuh"

namespace evo {

cudaError_t block_norm_fwd_bf16(const BlockNormCall& c, cudaStream_t st) {
  return norm::run_fwd<__nv_bfloat16, __nv_bfloat16>(c, st);
}

cudaError_t block_norm_bwd_bf16(const BlockNormCall& c, cudaStream_t st) {
  return norm::run_bwd<__nv_bfloat16, __nv_bfloat16>(c, st);
}

size_t block_norm_bwd_workspace_bytes(int C) {
  // the sums of every CTA, and at most kNormMaxItems pieces of shared gate rows
  return (size_t)(norm::kSums * kNormMaxCtas + kNormMaxItems) * C * sizeof(float);
}

}  // namespace evo
