// The block norm's kernels for: fp32 residual stream and block tensors.
#include "block_norm.cuh"

namespace evo {

cudaError_t block_norm_fwd_f32(const BlockNormCall& c, cudaStream_t st) {
  return norm::run_fwd<float, float>(c, st);
}

cudaError_t block_norm_bwd_f32(const BlockNormCall& c, cudaStream_t st) {
  return norm::run_bwd<float, float>(c, st);
}

}  // namespace evo
