// The block norm's kernels for: fp32 residual stream, bf16 block tensors.
#include "block_norm.cuh"

namespace evo {

cudaError_t block_norm_fwd_mixed(const BlockNormCall& c, cudaStream_t st) {
  return norm::run_fwd<float, __nv_bfloat16>(c, st);
}

cudaError_t block_norm_bwd_mixed(const BlockNormCall& c, cudaStream_t st) {
  return norm::run_bwd<float, __nv_bfloat16>(c, st);
}

}  // namespace evo
