// Launches: dynamic shared memory, and pairs of launches that overlap.
#pragma once

#include <atomic>

#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {

// An error that the caller returns to its own caller, not left behind in the runtime for
// the next call's look at its own launch.
inline cudaError_t taken(cudaError_t err) {
  if (err != cudaSuccess) (void)cudaGetLastError();
  return err;
}

// Lets a kernel have as much dynamic shared memory as the GPU holds beside its static
// one, once per device (the driver call takes a microsecond or two, a tenth of a small
// call).  Every caller sets the same limit, whatever it needs itself: of threads that
// come here together none can lower it for another.  Also below 48 KB: the static
// shared memory counts towards those too.  A launch that needs more than there is fails
// by itself.
template <auto Kernel>
cudaError_t allow_smem(size_t bytes) {
  static std::atomic<bool> done[64];
  if (bytes == 0) return cudaSuccess;
  int dev = 0, most = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return taken(err);
  if (dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  cudaFuncAttributes own;
  err = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (err == cudaSuccess) err = cudaFuncGetAttributes(&own, Kernel);
  if (err == cudaSuccess)
    err = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               most - (int)own.sharedSizeBytes);
  if (err != cudaSuccess) return taken(err);
  if (dev < 64) done[dev].store(true, std::memory_order_release);
  return cudaSuccess;
}

// Programmatic dependent launch.  The first kernel of a pair calls `let_second` as it
// begins; the second, launched with `launch_beside`, begins as the first's CTAs leave
// room, does what needs none of the first's results, and calls `wait_first` (the
// hardware's wait for the end of the first) before what does.
__device__ __forceinline__ void let_second() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_first() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename K, typename... A>
cudaError_t launch_beside(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream,
                          const A &...args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return taken(cudaLaunchKernelEx(&cfg, kernel, args...));
}

}  // namespace gdn
