// context_attention.h -- what the attention kernels over the paged cache
// share: their parameters, the split of a batch's work over the CTAs, and
// the joining of the parts of a split item.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dg.h"
#include "dg_device.cuh"

namespace dg {

struct AttnParams {
  // the batch (dg_context)
  const int32_t* table;
  const int32_t* lens;
  const int32_t* start;
  int32_t B, max_pages, pages, rows;
  // the cache
  const float* k_scale;
  const float* v_scale;
  int32_t kv_heads, group;  // group = query heads per kv head
  // queries and results
  const uint8_t* q;
  uint8_t* out;
  int64_t q_row, q_head, out_row, out_head;  // strides in bytes
  float* lse;
  float scale_log2;  // logit factor times log2(e)
  const uint8_t* causal;
  int32_t window;
  // workspace
  float* part;        // [2 * grid][part_floats]
  uint32_t* tickets;  // [grid], 0 between launches (rows kernel)
  void* splits;       // [grid] the split items (tiles kernel)
  uint32_t* err;
  uint64_t wait_ns;
  int32_t min_tiles;  // least tiles a CTA takes
};

// A request of the batch, as a kernel sees it: lengths a plan wrote, held
// within what the tables and rows can address.
struct Request {
  int row0, nq, len;
  bool causal;
};
DG_DEV Request request_of(const AttnParams& p, int r) {
  Request q;
  q.row0 = min(max(p.start[r], 0), p.rows);
  q.nq = max(min(p.start[r + 1], p.rows) - q.row0, 0);
  const int64_t room = static_cast<int64_t>(p.max_pages) * DG_PAGE;
  q.len = static_cast<int>(min(static_cast<int64_t>(max(p.lens[r], 0)), room));
  q.causal = p.causal != nullptr && p.causal[r] != 0;
  return q;
}

DG_DEV float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }  // -126 <= e <= 127

// The keys [lo, hi] that query row i (of nq) of a request sees.
DG_DEV int key_lo(const AttnParams& p, const Request& q, int i) {
  return p.window > 0 ? max(q.len - q.nq + i - p.window + 1, 0) : 0;
}
DG_DEV int key_hi(const Request& q, int i) { return q.causal ? q.len - q.nq + i : q.len - 1; }

// a / b of numbers that are not negative; 64-bit division, a routine of some
// hundred instructions, only where it takes 64 bits.
DG_DEV int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// Work is cut into tiles: kM packed query rows (row rho is query row rho /
// group, head rho % group of the kv head) by kKeys keys.  An item is one
// (request, row tile, kv head) with all key tiles that some row of it sees
// (one empty tile when none does, so that its zeros get written).  Items in
// order, each with its key tiles in order, form one line of tiles; every CTA
// takes an equal piece of that line (per = max(min_tiles, ceil(total /
// grid)) units), whatever requests it spans: ragged batches and single long
// contexts are split evenly by the same rule, and the rule follows the
// lengths alone.  An item is kCost units longer than its tiles, for what it
// costs beside them (queries, result): they lie ahead of its first tile, and
// nobody works on them.
template <int kM, int kKeys, int kCost>
struct Split {
  static DG_DEV int row_tiles(const AttnParams& p, const Request& q) {
    return static_cast<int>((static_cast<int64_t>(q.nq) * p.group + kM - 1) / kM);
  }
  static DG_DEV int item_tiles(const AttnParams& p, const Request& q, int mt, int* first) {
    const uint32_t rho = static_cast<uint32_t>(mt) * kM, group = static_cast<uint32_t>(p.group);  // rows * group is below 2^31
    const int i0 = static_cast<int>(rho / group);
    const int i1 = min(static_cast<int>((rho + kM - 1) / group), q.nq - 1);
    const int lo = key_lo(p, q, i0), hi = key_hi(q, i1);
    *first = hi >= lo ? lo / kKeys : 0;
    return hi >= lo ? hi / kKeys - lo / kKeys + 1 : 1;
  }
  // Sum over lanes of the tiles of row tiles mt0 + lane, mt0 + 32 + lane, ...
  static DG_DEV int64_t warp_tiles(const AttnParams& p, const Request& q, int mts) {
    int64_t n = 0;
    int f;
    for (int m = static_cast<int>(threadIdx.x & 31); m < mts; m += 32) n += item_tiles(p, q, m, &f);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
    return n;
  }
  // Fills before[0 .. B] (shared): tiles of the requests before r.  All
  // threads of the block; ends with a barrier.  A thread per request; the
  // requests whose row tiles differ in length (causal, window) and are many
  // get a warp each.
  static DG_DEV void totals(const AttnParams& p, int64_t* before) {
    for (int r = threadIdx.x; r < p.B; r += blockDim.x) {
      const Request q = request_of(p, r);
      const int mts = row_tiles(p, q);
      int64_t n = 0;
      int f;
      if (!q.causal && p.window == 0) {
        n = mts > 0 ? static_cast<int64_t>(mts) * item_tiles(p, q, 0, &f) : 0;
      } else if (mts <= 8) {
        for (int m = 0; m < mts; ++m) n += item_tiles(p, q, m, &f);
      } else {
        n = -1;
      }
      before[r + 1] = n < 0 ? n : (n + static_cast<int64_t>(mts) * kCost) * p.kv_heads;
    }
    if (threadIdx.x == 0) before[0] = 0;
    __syncthreads();
    for (int r = threadIdx.x >> 5; r < p.B; r += blockDim.x >> 5) {
      if (before[r + 1] >= 0) continue;  // the same for the whole warp
      const Request q = request_of(p, r);
      const int mts = row_tiles(p, q);
      const int64_t n = warp_tiles(p, q, mts) + static_cast<int64_t>(mts) * kCost;
      if ((threadIdx.x & 31) == 0) before[r + 1] = n * p.kv_heads;
    }
    __syncthreads();
    if (threadIdx.x < 32) {  // inclusive sums, 32 requests at a time
      int64_t carry = 0;
      for (int r0 = 0; r0 < p.B; r0 += 32) {
        const int r = r0 + threadIdx.x;
        int64_t v = r < p.B ? before[r + 1] : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int64_t o = __shfl_up_sync(0xffffffffu, v, d);
          if (static_cast<int>(threadIdx.x) >= d) v += o;
        }
        v += carry;
        if (r < p.B) before[r + 1] = v;
        carry = __shfl_sync(0xffffffffu, v, 31);
      }
    }
    __syncthreads();
  }

  int r, mt, h;          // the item
  Request q;
  int64_t begin;         // its first tile on the line (behind its cost)
  int tiles, first;      // its key tiles: first, first + 1, ...
  // The item that holds unit `pos` of the line.  All lanes of a warp, with the
  // same arguments.
  DG_DEV void find(const AttnParams& p, const int64_t* before, int64_t pos) {
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (before[mid + 1] > pos)
        hi = mid;
      else
        lo = mid + 1;
    }
    r = lo;
    q = request_of(p, r);
    begin = before[r];
    if (!q.causal && p.window == 0) {  // every row tile sees the same keys
      tiles = item_tiles(p, q, 0, &first);
      const int64_t n = quotient(pos - begin, tiles + kCost);
      mt = static_cast<int>(quotient(n, p.kv_heads));
      h = static_cast<int>(n - static_cast<int64_t>(mt) * p.kv_heads);
      begin += n * (tiles + kCost) + kCost;
      return;
    }
    const int lane = static_cast<int>(threadIdx.x & 31);
    const int mts = row_tiles(p, q);
    for (int m0 = 0;; m0 += 32) {  // 32 row tiles at a time
      int f = 0;
      const int n = m0 + lane < mts ? item_tiles(p, q, m0 + lane, &f) + kCost : 0;
      int64_t upto = static_cast<int64_t>(n) * p.kv_heads;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
      }
      const unsigned behind = __ballot_sync(0xffffffffu, begin + upto > pos);
      if (behind == 0 && m0 + 32 < mts) {
        begin += __shfl_sync(0xffffffffu, upto, 31);
        continue;
      }
      const int at = behind == 0 ? 31 : __ffs(behind) - 1;
      const int units = __shfl_sync(0xffffffffu, n, at);
      first = __shfl_sync(0xffffffffu, f, at);
      begin += __shfl_sync(0xffffffffu, upto, at) - static_cast<int64_t>(units) * p.kv_heads;
      mt = m0 + at;
      h = static_cast<int>(quotient(pos - begin, units));
      begin += static_cast<int64_t>(h) * units + kCost;
      tiles = units - kCost;
      return;
    }
  }
};

// The weight of a part whose logits are relative to 2^m when parts are joined
// relative to 2^top.
DG_DEV float join_weight(float m, float top) { return exp2f(m - top); }

DG_DEV float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The kernel for many rows (context_tiles.cu): its resident CTAs on the
// current device (-1: none), the floats of one part, the bytes of one split
// item, its launch.
int tiles_grid(int dim);
size_t tiles_part_floats(int dim);
size_t tiles_split_bytes();
cudaError_t launch_attention_tiles(int dim, const CUtensorMap& tmK, const CUtensorMap& tmV, const AttnParams& p,
                                   int grid, cudaStream_t stream);

}  // namespace dg
