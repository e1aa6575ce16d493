// fa_cache_launch.cuh -- host helpers that the cache kernels' launchers share.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "fa_device.h"

namespace fa {

// Once per kernel and device: its shared memory.
template <class K>
bool allow_smem(K kern, int bytes, int dev, std::atomic<unsigned long long>& configured) {
  if ((configured.load(std::memory_order_acquire) >> dev) & 1ull) return true;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) {
    set_error("cudaFuncSetAttribute(max dynamic smem = %d): %s", bytes, cudaGetErrorString(e));
    return false;
  }
  configured.fetch_or(1ull << dev, std::memory_order_release);
  return true;
}

// Programmatic launch: the blocks come up while the kernel before ends, and
// wait for it (griddepcontrol.wait) before they read what it wrote.
template <class... P>
cudaError_t launch_after(void (*kern)(P...), dim3 grid, unsigned threads, cudaStream_t stream, const P&... p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p...);
}

}  // namespace fa
