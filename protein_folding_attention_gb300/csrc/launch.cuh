// Launches that overlap the end of the kernel before them.
#pragma once
#include <cuda_runtime.h>

namespace evo {

// First thing in a kernel launched by launch_early: waits until the work
// before it in the stream has ended and its writes are visible.
__device__ __forceinline__ void wait_for_earlier_work() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets a next launch of that kind be set up; it still waits for this kernel.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A launch whose set-up may overlap the end of the kernel before it in the
// stream.  The kernel calls wait_for_earlier_work before it reads or writes
// global memory.
template <typename K, typename... A>
cudaError_t launch_early(K kernel, unsigned grid, unsigned threads, size_t smem, cudaStream_t st,
                         const A&... args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace evo
