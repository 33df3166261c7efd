// Launchers of the optimiser kernels (evoattn_grad_norm, evoattn_adamw).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>

#include "evoattn.h"

namespace evo {

struct AdamwScalars {
  float lr;
  const float* lr_device;
  double beta1, beta2;
  float eps;
  bool clip;
};

size_t grad_norm_workspace_bytes(int count);
cudaError_t grad_norm(const evoattn_adamw_tensor* t, int count, float max_norm,
                      evoattn_optim_state* state, void* ws, cudaStream_t st);
cudaError_t adamw32(const evoattn_adamw_tensor* t, int count, const AdamwScalars& s,
                    evoattn_optim_state* state, cudaStream_t st);
cudaError_t adamw8(const evoattn_adamw_tensor* t, int count, const AdamwScalars& s,
                   evoattn_optim_state* state, cudaStream_t st);

}  // namespace evo
