// What a launch needs of the current device, asked for once a device instead of at every call.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace gcs {

// The current device's number, -1 on an error.
inline int current_device() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess ? dev : -1;
}

// SMs of the current device, 0 on an error.
inline int current_sms() {
  static std::atomic<int> known[64];
  const int dev = current_device();
  if (dev < 0) return 0;
  int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (!n) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Lets a kernel take up to `bytes` of dynamic shared memory on the current device; the largest size
// of all calls has to be asked for (it is set once a device, or again where it grew).
template <auto Kernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<int> set[64];
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (dev < 64 && set[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) set[dev].store(bytes, std::memory_order_relaxed);
  return e;
}

#ifdef __CUDACC__
// In a kernel that may run beside the one before it: what comes after it waits for it alone, so none of
// its blocks ends before that one has.
struct WaitAtEnd {
  __device__ __forceinline__ ~WaitAtEnd() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
};
#endif

// Launches a kernel that may start while the stream's kernel before it still runs (once that one has
// let it, or has ended): it waits by itself for what it needs of it, or needs nothing.
template <typename... Args, typename... Given>
cudaError_t launch_beside(void (*kern)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t s, Given... given) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, given...);
}

}  // namespace gcs
