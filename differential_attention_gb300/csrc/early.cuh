// early.cuh -- programmatic launches: a kernel is set up while the one before it in the stream still runs.
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace da {

// Until the kernels before this one are done and their writes seen (by plain loads: what they wrote was not
// constant while this kernel ran, so nothing of it is read through __ldg). Every block of a kernel that is
// launched this way calls it, also one that has nothing to do: the kernel after it goes by that.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// From here on (in all blocks) the kernel after this one may be set up. After grid_wait().
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Whether this file's kernels were ever launched: until then its status word is 0 and need not be read.
static std::atomic<bool> g_launched{false};

// This file's status word; cleared where it is set.
static inline cudaError_t launched_status(int* v) {
  if (!g_launched.load(std::memory_order_relaxed)) return cudaSuccess;
  cudaError_t e = cudaMemcpyFromSymbol(v, g_device_status, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess && *v != 0) e = cudaMemcpyToSymbol(g_device_status, &zero, sizeof(int));
  return e;
}

// Launches a kernel that calls grid_wait() first: it is set up while the one before it in the stream ends.
template <typename P>
static cudaError_t launch_early(void (*kernel)(P), unsigned grid, int block, int smem, cudaStream_t st, int cluster,
                                const P& p) {
  g_launched.store(true, std::memory_order_relaxed);
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// launch_early of a kernel with more than 48 KB of dynamic shared memory (at most `limit`). The limit is
// raised on each device's first call (`raised`: a bit each), and again where a launch is refused, as
// after a reset of the device.
template <typename P>
static cudaError_t launch_early_large(void (*kernel)(P), unsigned grid, int block, int smem, int limit, cudaStream_t st,
                                      int cluster, const P& p, std::atomic<uint64_t>& raised) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (raised.load(std::memory_order_relaxed) & bit) {
    e = launch_early(kernel, grid, block, smem, st, cluster, p);
    if (e != cudaErrorInvalidValue) return e;
    cudaGetLastError();
  }
  e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize, limit);
  if (e != cudaSuccess) return e;
  raised.fetch_or(bit, std::memory_order_relaxed);
  return launch_early(kernel, grid, block, smem, st, cluster, p);
}

}  // namespace da
