// Host and device sides of launches: what a kernel needs before its first one, and launches that may
// begin before the kernel in front of them has ended.
#pragma once
#include <cuda_runtime.h>

#include <atomic>

namespace fa {

__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Lets a kernel use `bytes` of dynamic shared memory on the current device, and checks that
// it has at least `regs` registers a thread; once per device (a bit each of `ready`).
inline cudaError_t allow_smem(const void* kern, int bytes, int regs,
                              std::atomic<unsigned long long>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (ready.load(std::memory_order_acquire) & bit) return cudaSuccess;
  cudaFuncAttributes attr;
  if ((e = cudaFuncGetAttributes(&attr, kern)) != cudaSuccess) return e;
  if (attr.numRegs < regs) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_release);
  return e;
}

// Launches what follows a kernel just launched on `stream`. It may be scheduled while that
// one runs; its blocks wait for its end (pdl_wait) before they read anything.
template <typename... P, typename... A>
cudaError_t launch_next(void (*kern)(P...), dim3 grid, int threads, int smem, cudaStream_t stream,
                        const A&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// The merge of a kernel's pieces.
template <typename... P, typename... A>
cudaError_t launch_merge(void (*kern)(P...), dim3 grid, int threads, cudaStream_t stream,
                         const A&... args) {
  return launch_next(kern, grid, threads, 0, stream, args...);
}

}  // namespace fa
