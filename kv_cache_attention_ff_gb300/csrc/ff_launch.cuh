// Launches that overlap the end of the kernel before them, and what the caches' kernels share besides.
#pragma once

#include <cstddef>
#include <cuda_runtime.h>

namespace ff {

// The caches' kernels are launched so that one may start before the one ahead of it on
// the stream has ended (launch_kernel): grid_wait() stands before the first
// access to memory that another kernel may write or read, and returns when all
// earlier work is complete.  What it hides is the launch itself, some 2 us.
// Memory that those kernels write is read with plain or __ldcg loads: __ldg and
// ld.global.nc take it as constant while the kernel runs, and may be moved
// before the wait.
__device__ __forceinline__ void grid_wait() {
  asm volatile("griddepcontrol.launch_dependents;\n griddepcontrol.wait;" ::: "memory");
}

template <class... P, class... A>
cudaError_t launch_kernel(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s, int cluster,
                          const A&... args) {
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

}  // namespace ff
