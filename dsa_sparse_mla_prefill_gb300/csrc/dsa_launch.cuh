// A launch whose start may overlap the end of the kernel before it on the stream.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace dsa {

// Programmatic stream serialization: the grid may be put on the GPU once every CTA of
// the kernel before has ended or called launch_dependents().  Such a kernel calls
// wait_for_previous() before it touches global memory, and reads it with plain loads:
// the read-only path (__ldg) wants memory that nobody writes while the kernel is
// there, and the compiler may move such a load above the wait.
template <typename... P, typename... A>
static int launch_after(void (*kernel)(P...), dim3 grid, int threads, uint32_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess) return 0;
  cudaGetLastError();   // (reported here, not by the next launch)
  return -1;
}

// Lets a kernel have `smem` bytes of dynamic shared memory on the current device.  done:
// the kernel's own, zeros at first, so that the devices it was asked for once are not
// asked again.
static inline int allow_smem(const void* kernel, uint32_t smem, int (&done)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess) {
    if (dev < 64 && done[dev]) return 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess) {
      if (dev < 64) done[dev] = 1;
      return 0;
    }
  }
  cudaGetLastError();   // (reported here, not by the next launch)
  return -1;
}

__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace dsa
