// pa_launch.h - kernel launches in clusters (not part of the public ABI).
#pragma once

#include <atomic>

#include "pa_internal.h"

namespace pa {

// A kernel whose warps raise their register limits (setmaxnreg) out of the `regs` registers that a thread is launched
// with: built with fewer (a debug build, another compiler's choice), the warps would wait for registers that no one
// gives back, for ever, so it is not launched.  `known`: the kernel has been looked at.
inline cudaError_t require_registers(const void* kernel, int regs, std::atomic<bool>& known) {
  if (known.load(std::memory_order_relaxed)) return cudaSuccess;
  cudaFuncAttributes a;
  const cudaError_t e = cudaFuncGetAttributes(&a, kernel);
  if (e != cudaSuccess) return e;
  if (a.numRegs < regs) return cudaErrorInvalidConfiguration;
  known.store(true, std::memory_order_relaxed);
  return cudaSuccess;
}

// Launch in clusters of `cluster` CTAs (1: none), as a programmatic dependent of the kernel before it (see
// launch_dependent) if `dependent`.
template <typename... Params, typename... Args>
inline cudaError_t launch_cluster(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, int cluster,
                                  bool dependent, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (dependent) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)cluster;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = (unsigned)n;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace pa
