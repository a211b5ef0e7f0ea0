// pdl.h -- launch with programmatic stream serialization: the grid may start before the
// previous kernel on its stream has finished, and the kernel waits (grid_dependency_wait in
// ptx.cuh) before it touches global memory. Errors are left for cudaGetLastError.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace gemm_gb300 {

template <typename... P, typename... A>
void launch_pdl(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A &&...args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(std::forward<A>(args))...);
}

}  // namespace gemm_gb300
