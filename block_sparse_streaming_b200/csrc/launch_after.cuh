// launch_after.cuh - launch of a kernel that overlaps the end of the one before it.
#pragma once

#include <cuda_runtime.h>

namespace loza {

// A kernel behind the one that writes what it reads (it waits for it itself).
template <typename P>
bool launch_after(void (*kernel)(P), dim3 grid, unsigned threads, cudaStream_t st, const P& prm) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, prm) == cudaSuccess;
}

}  // namespace loza
