// context.h -- what the context entry points (context.cu,
// context_attention.cu) share on the host side.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dg.h"

namespace dg {

// Rows of one batch: keeps row, run and tile numbers in 32 bits.
constexpr int kContextMaxRows = 1 << 24;

// The argument checks of the context entry points.
dg_status check_context(const dg_context* c);
dg_status check_heads(const dg_heads* t, int heads, int dim);
dg_status check_cache(const dg_context_cache* c, const dg_context* ctx);

// Launch as a programmatic dependent of the kernel before: the blocks of a
// context kernel come up, and set up what needs no input, while that one
// ends.  Every context kernel waits for its predecessors before its first
// access to global memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_context(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                           Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, KArgs(args)...);
}

}  // namespace dg
