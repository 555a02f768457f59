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

}  // namespace dg
