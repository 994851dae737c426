// Launches that may begin while the kernel before them in the stream still runs: the set-up of one
// kernel overlaps the end of the other.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moe.h"

namespace dsv4 {

// In a kernel that was launched so: waits for all that is before it in the stream.  The next one
// may be launched from here on (it waits in its turn).
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

inline int sm_count() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 148;
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), int64_t grid, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
  if (e == cudaSuccess)
    note_launch(1);
  else
    (void)cudaGetLastError();  // returned here, and not by a later call that asks for the last error
  return e;
}

}  // namespace dsv4
