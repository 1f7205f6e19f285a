// Launches whose blocks may start while the stream's kernel before is ending: they
// set up, then wait for its end and its writes (launched_after) before they touch
// global memory.  Every block waits, also one without work, so that a kernel never
// ends before the one that it was launched after; the library's other kernels that
// are launched so (joins, second kernels of a call) keep to that too.  (Calls in a row
// on one GB300: a product of 8 tokens 4.6 -> 4.2 us in a graph, 6.2 -> 4.1 without, a
// prompt of 256 12.1 -> 8.1.  Letting the next kernel start while this one still works
// gave 0.1 us there and took 1.5 here.)
#pragma once

#include <cuda_runtime.h>

#include "mla_layer_ops.h"

namespace mtv {

__device__ __forceinline__ void launched_after() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The count of MTV_TEST_GIVE_UP in a dtype argument, which is left without it; what is none stays as it is.
inline int take_give_up(int* dtype) {
  if (*dtype < 0 || *dtype >= 256 * MTV_TEST_GIVE_UP) return 0;
  const int n = *dtype / MTV_TEST_GIVE_UP;
  *dtype %= MTV_TEST_GIVE_UP;
  return n;
}

template <typename... P>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, const P&... args) {
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config = {};
  config.gridDim = grid;
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = smem;
  config.stream = st;
  config.attrs = early;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, args...);
}

}  // namespace mtv
