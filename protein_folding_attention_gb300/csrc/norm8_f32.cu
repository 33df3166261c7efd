// The residual add with dropout and the norm with 8-bit output for: fp32 residual stream,
// fp32 block tensors.
#include "norm8.cuh"

namespace evo {

cudaError_t dropout_add_f32(const Norm8Call& c, cudaStream_t st) { return norm8::run_dropout<float, float>(c, st); }
cudaError_t norm8_fwd_f32(const Norm8Call& c, cudaStream_t st) { return norm8::run_fwd<float, float>(c, st); }
cudaError_t norm8_bwd_f32(const Norm8Call& c, cudaStream_t st) { return norm8::run_bwd<float, float>(c, st); }

}  // namespace evo
