// The residual add with dropout and the norm with 8-bit output for: fp32 residual stream,
// bf16 block tensors (and the dropout from fp32 to bf16).
#include "norm8.cuh"

namespace evo {

cudaError_t dropout_add_mixed(const Norm8Call& c, cudaStream_t st) { return norm8::run_dropout<float, __nv_bfloat16>(c, st); }
cudaError_t dropout_add_narrow(const Norm8Call& c, cudaStream_t st) {
  return norm8::run_dropout<__nv_bfloat16, float>(c, st);
}
cudaError_t norm8_fwd_mixed(const Norm8Call& c, cudaStream_t st) { return norm8::run_fwd<float, __nv_bfloat16>(c, st); }
cudaError_t norm8_bwd_mixed(const Norm8Call& c, cudaStream_t st) { return norm8::run_bwd<float, __nv_bfloat16>(c, st); }

}  // namespace evo
