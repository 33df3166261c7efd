// The residual add with dropout and the norm with 8-bit output for: bf16 residual stream,
// bf16 block tensors.
#include "norm8.cuh"

namespace evo {

cudaError_t dropout_add_bf16(const Norm8Call& c, cudaStream_t st) { return norm8::run_dropout<__nv_bfloat16, __nv_bfloat16>(c, st); }
cudaError_t norm8_fwd_bf16(const Norm8Call& c, cudaStream_t st) { return norm8::run_fwd<__nv_bfloat16, __nv_bfloat16>(c, st); }
cudaError_t norm8_bwd_bf16(const Norm8Call& c, cudaStream_t st) { return norm8::run_bwd<__nv_bfloat16, __nv_bfloat16>(c, st); }

size_t norm8_bwd_workspace_bytes(int C) { return (size_t)2 * kNorm8MaxCtas * C * sizeof(float); }

}  // namespace evo
