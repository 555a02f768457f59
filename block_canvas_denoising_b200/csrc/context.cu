// context.cu -- the context of block-by-block generation: block tables and
// slot maps from request lengths, rotary positions, and the append of keys
// and values to the 8-bit paged cache ("DiffusionGemma Technical Report",
// Figure 4: each finished block is encoded and appended to the context the
// next block is conditioned on).  The attention over the cache is
// context_attention.cu.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <math.h>
#include <stdio.h>

#include "context.h"
#include "dg_device.cuh"
#include "dg_internal.h"

namespace dg {

namespace {

// ---------------------------------------------------------------------------
// block tables and slot maps
// ---------------------------------------------------------------------------
constexpr int kPlanCtas = 8;  // one cluster
constexpr int kPlanThreads = 256;
static_assert(kPlanThreads >= DG_MAX_B, "one thread per request");

// Exclusive prefix sums over the block's threads of four values at once.
struct Quad {
  int64_t v[4];
};
DG_DEV Quad block_prefix(Quad x, Quad* total, Quad* warp_sums /* [8] shared */) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Quad inc = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int64_t o = __shfl_up_sync(0xffffffffu, inc.v[c], d);
      if (lane >= d) inc.v[c] += o;
    }
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  Quad before = {}, all = {};
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (w < warp) before.v[c] += warp_sums[w].v[c];
      all.v[c] += warp_sums[w].v[c];
    }
  }
  *total = all;
#pragma unroll
  for (int c = 0; c < 4; ++c) before.v[c] += inc.v[c] - x.v[c];
  __syncthreads();
  return before;
}

// The request whose half-open range [start[r], start[r + 1]) holds i.
DG_DEV int owner_of(const int* start, int B, int i) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (start[mid + 1] > i)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// One cluster plans the batch.  Every CTA reads the lengths (one thread per
// request) and forms the same prefix sums: pages given back, pages needed,
// rows and runs before each request.  The tables, rows and runs are then
// written by all CTAs together.  Nothing here is bandwidth: 12 bytes a row
// and 16 a run.  What it costs is the chain of dependent reads (lengths, the
// stack, the table) and the two cluster barriers that keep every read of the
// old state before the first write of the new one; one launch with barriers
// in hardware instead of three launches in a row.  8 requests x 256 rows take
// 4.5 us in a graph of their own and 3.0 one after another, 256 requests x up to
// 300 rows with some leaving 8.6 and 6.8 (18.7 with a search per row instead of
// per run).
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
context_plan_kernel(const dg_context c, const int32_t* __restrict__ add, const uint8_t* __restrict__ release,
                    int32_t commit) {
  __shared__ Quad sums[kPlanThreads / 32];
  __shared__ int s_held[DG_MAX_B], s_gone0[DG_MAX_B], s_gone[DG_MAX_B], s_need0[DG_MAX_B], s_need[DG_MAX_B];
  __shared__ int s_start[DG_MAX_B + 1], s_run0[DG_MAX_B + 1];
  __shared__ int s_bad;
  const int tid = threadIdx.x;
  const int rank = static_cast<int>(cluster_ctarank());
  const int gtid = rank * kPlanThreads + tid, gsize = kPlanCtas * kPlanThreads;
  const int B = c.B;
  const int64_t room = static_cast<int64_t>(c.max_pages) * DG_PAGE;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  wait_for_previous_kernel();
  allow_next_kernel();

  // nothing here reads it: first, and by a thread with little to do (by the one
  // that writes the results, at the end, plans took 0.1 to 0.3 us more)
  if (rank == kPlanCtas - 1 && tid == kPlanThreads - 1 && c.epoch != nullptr) atomicAdd(c.epoch, 1);
  const int64_t free0 = *(commit ? c.free_next : c.free_count);
  int64_t held = 0, a = 0, gone = 0, need = 0, touched = 0;
  if (tid < B) {
    held = commit ? c.lens[tid] : c.held[tid];
    a = add[tid];
    bool bad = held < 0 || held > room || a < 0;
    if (!bad && release != nullptr && release[tid]) {
      gone = (held + DG_PAGE - 1) / DG_PAGE;
      held = 0;
    }
    bad = bad || held + a > room;
    if (bad) {
      s_bad = 1;
      a = 0;
    }
    need = (held + a + DG_PAGE - 1) / DG_PAGE - (held + DG_PAGE - 1) / DG_PAGE;
    touched = a > 0 ? (held + a - 1) / DG_PAGE - held / DG_PAGE + 1 : 0;
  }
  Quad tot;
  const Quad pre = block_prefix(Quad{{gone, need, a, touched}}, &tot, sums);
  const bool stack_bad = free0 < 0 || free0 + tot.v[0] > c.pages;
  const int64_t free1 = free0 + tot.v[0];
  const int code = (s_bad || stack_bad) ? 3 : tot.v[2] > c.rows ? 2 : tot.v[1] > free1 ? 1 : 0;
  const bool ok = code == 0;
  if (tid < B) {
    s_held[tid] = static_cast<int>(held);
    s_gone0[tid] = static_cast<int>(pre.v[0]);
    s_gone[tid] = stack_bad ? 0 : static_cast<int>(gone);
    s_need0[tid] = ok ? static_cast<int>(pre.v[1]) : 0;
    s_need[tid] = ok ? static_cast<int>(need) : 0;
    s_start[tid] = ok ? static_cast<int>(pre.v[2]) : 0;
    s_run0[tid] = ok ? static_cast<int>(pre.v[3]) : 0;
  }
  if (tid == 0) {
    s_start[B] = ok ? static_cast<int>(tot.v[2]) : 0;
    s_run0[B] = ok ? static_cast<int>(tot.v[3]) : 0;
  }
  cluster_sync_all();  // every CTA has read held, lens and the stack's height

  const int warp = gtid >> 5, lane = tid & 31, warps = gsize >> 5;
  if (release != nullptr) {
    for (int r = warp; r < B; r += warps)
      for (int j = lane; j < s_gone[r]; j += 32)
        c.free_list[free0 + s_gone0[r] + j] = c.table[static_cast<size_t>(r) * c.max_pages + j];
    __threadfence();
    cluster_sync_all();  // the pages given back are on the stack
  }

  const int total = s_start[B];
  // page j of request r: held pages stand in the table, new ones on the stack
  auto page_of = [&](int r, int j) {
    const int first = (s_held[r] + DG_PAGE - 1) / DG_PAGE;
    return j < first ? c.table[static_cast<size_t>(r) * c.max_pages + j]
                     : c.free_list[free1 - 1 - s_need0[r] - (j - first)];
  };
  // Rows by their runs: a lane finds one run's request and page (a search and
  // a read, 32 of them at once), and the warp then writes the rows of each.
  const int runs = DG_CONTEXT_RUNS(c.rows, B), used = s_run0[B];
  for (int u0 = warp; u0 < runs; u0 += 32 * warps) {
    const int u = u0 + lane * warps;
    int4 run = make_int4(-1, 0, 0, 0);
    int pos = 0;
    if (u < used) {
      const int r = owner_of(s_run0, B, u);
      const int h = s_held[r], end = h + s_start[r + 1] - s_start[r];
      const int j = h / DG_PAGE + u - s_run0[r];
      const int lo = max(j * DG_PAGE, h), hi = min((j + 1) * DG_PAGE, end);
      run = make_int4(page_of(r, j), s_start[r] + lo - h, lo - j * DG_PAGE, hi - lo);
      pos = lo;
    }
    if (u < runs) reinterpret_cast<int4*>(c.runs)[u] = run;
    const int n = min(32, (used - u0 + warps - 1) / warps);  // runs the warp has in hand
    for (int k = 0; k < n; ++k) {
      const int page = __shfl_sync(0xffffffffu, run.x, k), row = __shfl_sync(0xffffffffu, run.y, k);
      const int off = __shfl_sync(0xffffffffu, run.z, k), count = __shfl_sync(0xffffffffu, run.w, k);
      const int first = __shfl_sync(0xffffffffu, pos, k);
      for (int i = lane; i < count; i += 32) {
        c.positions[row + i] = first + i;
        c.slots[row + i] = static_cast<int64_t>(page) * DG_PAGE + off + i;
      }
    }
  }
  for (int i = total + gtid; i < c.rows; i += gsize) {
    c.positions[i] = -1;
    c.slots[i] = -1;
  }
  for (int r = warp; r < B; r += warps) {
    const int first = (s_held[r] + DG_PAGE - 1) / DG_PAGE;
    for (int j = lane; j < s_need[r]; j += 32)
      c.table[static_cast<size_t>(r) * c.max_pages + first + j] = c.free_list[free1 - 1 - s_need0[r] - j];
  }
  if (rank == 0) {
    if (tid < B) {
      c.held[tid] = s_held[tid];
      c.lens[tid] = s_held[tid] + s_start[tid + 1] - s_start[tid];
      c.start[tid] = s_start[tid];
    }
    if (tid == 0) {
      const int kept = static_cast<int>(stack_bad ? free0 : free1);
      c.start[B] = total;
      c.free_count[0] = kept;
      c.free_next[0] = kept - (ok ? static_cast<int>(tot.v[1]) : 0);
      c.status[0] = code;
    }
  }
}

// ---------------------------------------------------------------------------
// rotary positions
// ---------------------------------------------------------------------------
// A frequency as a fraction of a turn per position, in units of 2^-64: then
// position * turn, mod 2^64, is the exact place within a turn of a frequency
// that is off by at most 2^-64 + 2^-53 of itself (a float32 product is off by
// more than a hundredth of a radian at positions in the hundred thousands).
DG_DEV uint64_t turn_fraction(double freq) {
  double f = freq * 0.15915494309189533577;  // 1 / (2 pi)
  f -= floor(f);
  const uint32_t hi = static_cast<uint32_t>(f * 4294967296.0);  // f < 1
  const uint32_t lo = static_cast<uint32_t>((f * 4294967296.0 - hi) * 4294967296.0);
  return static_cast<uint64_t>(hi) << 32 | lo;
}
// (cos, sin) of a place within a turn, times the magnitude.  The nearest
// quarter turn goes off by integer arithmetic, and the rest, at most pi / 4,
// through the Taylor polynomials of degree 9 and 8, whose remainders there are
// (pi/4)^11 / 11! = 2e-9 and (pi/4)^10 / 10! = 3e-8, half a float32 step of 1.
DG_DEV float2 turn_of(uint64_t place, float magnitude) {
  const uint32_t p = static_cast<uint32_t>(place >> 32);
  const uint32_t quarter = (p + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(p - (quarter << 30))) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  const float z = x * x;
  float s = fmaf(z, 2.7557319223985893e-6f, -1.9841269841269841e-4f);
  s = fmaf(z, s, 8.3333333333333333e-3f);
  s = fmaf(z, s, -0.16666666666666667f);
  s = fmaf(z * x, s, x);
  float c = fmaf(z, 2.4801587301587302e-5f, -1.3888888888888889e-3f);
  c = fmaf(z, c, 4.1666666666666667e-2f);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.0f);
  const float co = (quarter & 1) ? s : c, si = (quarter & 1) ? c : s;
  // quarters: (c, s), (-s, c), (-c, -s), (s, -c)
  return make_float2((quarter == 1 || quarter == 2) ? -co * magnitude : co * magnitude,
                     (quarter == 2 || quarter == 3) ? -si * magnitude : si * magnitude);
}

DG_DEV void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
DG_DEV uint4 pack8(const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 o = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&o);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// A head is cut into units of two chunks of 8 elements, 16 units of work per
// 2 x 128 bytes: unit u < rot / 16 rotates with frequencies 8u .. 8u + 7 --
// chunks (u, u + rot / 16) hold the halves' partners, chunks (2u, 2u + 1)
// the interleaved pairs -- and every other unit is chunks (2u, 2u + 1) as
// they are.
DG_DEV void unit_chunks(int u, int rot16, bool interleaved, int& ca, int& cb) {
  const bool halves = u < rot16 && !interleaved;
  ca = halves ? u : 2 * u;
  cb = halves ? u + rot16 : 2 * u + 1;
}
// (x, y) turned.  Its roundings are spelled out, so that a number is the same
// wherever this is inlined.
DG_DEV void rotate_pair(float& x, float& y, const float2& t) {
  const float a = x, b = y;
  x = __fmaf_rn(a, t.x, -__fmul_rn(b, t.y));
  y = __fmaf_rn(a, t.y, __fmul_rn(b, t.x));
}
DG_DEV void rotate_unit(float (&a)[8], float (&b)[8], const float2 (&t)[8], bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rotate_pair(a[2 * i], a[2 * i + 1], t[i]);
      rotate_pair(b[2 * i], b[2 * i + 1], t[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) rotate_pair(a[i], b[i], t[i]);
  }
}

// Where the turn of frequency j = 8 u + 2 k + w lies in a token's row of turns,
// `units` units long: pair k of all units side by side, so that neighbouring
// threads (units) read neighbouring 16 bytes.
DG_DEV int turn_place(int j, int units) { return (((j >> 1) & 3) * units + (j >> 3)) * 2 + (j & 1); }
// The eight turns of unit u.
DG_DEV void read_turns(const float2* row, int u, int units, float2 (&t)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    *reinterpret_cast<float4*>(&t[2 * k]) = *reinterpret_cast<const float4*>(&row[(k * units + u) * 2]);
}

constexpr int kRopeThreads = 256;

// kTokens token rows per CTA.  The turns of a token serve all of its heads:
// they are formed once, by one thread per (token, frequency), and kept in
// shared memory; the heads then stream through, 32 bytes a thread, a thread
// staying on its unit and walking the (token, head) pairs by a fixed stride
// (256 threads / units = step_tokens * heads + step_heads) without a division.
// Bound by memory: 67 MB of 8191 rows x 16 heads x 128 take 13.4 us from HBM,
// 5.0 TB/s, 0.76 of a plain copy's rate (12.6 us with the input in L2).
template <int kDim, int kTokens>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(const uint8_t* x, uint8_t* out, int64_t xr, int64_t xh, int64_t outr, int64_t outh, int rows, int heads,
            int step_tokens, int step_heads, const int32_t* __restrict__ positions, const double* __restrict__ freq,
            int rot, int interleaved, float magnitude) {
  constexpr int kUnits = kDim / 16;                 // units per head
  __shared__ __align__(16) float2 turns[kTokens][kDim / 2];
  __shared__ int s_pos[kTokens];
  const int row0 = blockIdx.x * kTokens;
  const int half = rot / 2, rot16 = rot / 16;
  const int u = threadIdx.x % kUnits;
  int ca, cb;
  unit_chunks(u, rot16, interleaved, ca, cb);
  const bool turned = u < rot16, idle = x == out && !turned;
  const int tokens = min(kTokens, rows - row0);
  x += 2 * row0 * xr;
  out += 2 * row0 * outr;
  // this thread's first pair
  int token = 0, head = threadIdx.x / kUnits;
  while (head >= heads) {
    head -= heads;
    ++token;
  }
  auto next = [&](int& t, int& h) {
    t += step_tokens;
    h += step_heads;
    if (h >= heads) {
      h -= heads;
      ++t;
    }
  };
  auto load = [&](int t, int h, uint4& a, uint4& b) {
    const uint8_t* src = x + 2 * (t * xr + h * xh);
    a = *reinterpret_cast<const uint4*>(src + 16 * ca);
    b = *reinterpret_cast<const uint4*>(src + 16 * cb);
  };
  wait_for_previous_kernel();
  allow_next_kernel();
  // the first two are on their way while the turns are formed
  uint4 wa[2], wb[2];
  {
    int t = token, h = head;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (t < tokens && !idle) load(t, h, wa[k], wb[k]);
      next(t, h);
    }
  }
  for (int i = threadIdx.x; i < tokens * half; i += kRopeThreads) {
    const int t = i / half, j = i - t * half;
    turns[t][turn_place(j, rot16)] =
        turn_of(static_cast<uint32_t>(positions[row0 + t]) * turn_fraction(freq[j]), magnitude);
  }
  if (threadIdx.x < kTokens) s_pos[threadIdx.x] = threadIdx.x < tokens ? positions[row0 + threadIdx.x] : -1;
  __syncthreads();
  if (idle) return;
  for (int k = 0; token < tokens; k ^= 1) {
    uint4 va = k ? wa[1] : wa[0], vb = k ? wb[1] : wb[0];
    {  // the one after the next
      int t = token, h = head;
      next(t, h);
      next(t, h);
      if (t < tokens) {
        if (k)
          load(t, h, wa[1], wb[1]);
        else
          load(t, h, wa[0], wb[0]);
      }
    }
    if (s_pos[token] >= 0) {
      if (turned) {
        float a[8], b[8];
        unpack8(va, a);
        unpack8(vb, b);
        float2 tr[8];
        read_turns(turns[token], u, rot16, tr);
        rotate_unit(a, b, tr, interleaved);
        va = pack8(a);
        vb = pack8(b);
      }
      uint8_t* dst = out + 2 * (token * outr + head * outh);
      *reinterpret_cast<uint4*>(dst + 16 * ca) = va;
      *reinterpret_cast<uint4*>(dst + 16 * cb) = vb;
    }
    next(token, head);
  }
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
// The exponent of the least power of two s with top <= 448 s, at least -100;
// 0 for top = 0.  448 = 1.75 * 2^8, so with top = 1.m 2^E it is E - 8, and one
// more where 1.m is above 1.75 (a top that is subnormal ends at -100 anyway).
DG_DEV int scale_exponent(float top) {
  if (top == 0.f) return 0;
  const uint32_t b = __float_as_uint(top);
  return max(static_cast<int>(b >> 23) - 135 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0), -100);
}
DG_DEV float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }  // -126 <= e <= 127
// Two floats to E4M3, to nearest even, saturating; NaN stays NaN.
DG_DEV uint32_t e4m3_pair(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
DG_DEV uint2 e4m3_chunk(const float (&x)[8], float inv) {
  return make_uint2(e4m3_pair(x[0] * inv, x[1] * inv) | e4m3_pair(x[2] * inv, x[3] * inv) << 16,
                    e4m3_pair(x[4] * inv, x[5] * inv) | e4m3_pair(x[6] * inv, x[7] * inv) << 16);
}

// ---- held tokens on a page that a provisional batch goes on filling
// A batch may be planned over, and then the held codes it had rounded again
// must be there as they were.  They are few -- one page a request at most -- so
// they are put aside when the scale grows, in a place of the page's own
// (`pages` up to DG_MAX_B) or of its request's, with a tag that says of which
// page, which tokens and which plan they are, and what the append left in the
// page.  The next plan's append begins with them if the page is still that.  A
// mark beside each scale says in which plan and behind how many tokens it has
// grown, 0 if it has not since the page was begun: all that an append reads
// where nothing is to be done.
// (With every head's tag read in any case, 32 requests x 8 heads x 1 row took
// 3.8 us instead of 3.5.)
struct KeptTag {
  int32_t page, off;    // held tokens [0, off) of this page; off = 0: nothing
  uint32_t epoch;       // the plan whose batch made the scale grow
  float base, grown;    // scales before and after
  uint32_t check[2];    // sums over the codes as rounded again
};
DG_DEV uint32_t grown_mark(uint32_t epoch, int off) { return epoch << 6 | static_cast<uint32_t>(off); }  // off < DG_PAGE
// dg_context_cache.kept: marks [k, v][pages][heads], tags and codes [slots][k, v][heads].
DG_DEV uint32_t* kept_marks(const dg_context_cache& cache, bool is_k) {
  return reinterpret_cast<uint32_t*>(cache.kept) + (is_k ? 0 : static_cast<size_t>(cache.pages) * cache.heads);
}
struct KeptLayout {
  int slots;
  size_t tags, codes, total;
};
inline __host__ __device__ KeptLayout kept_layout(int pages, int heads, int dim) {
  KeptLayout l;
  l.slots = pages < DG_MAX_B ? pages : DG_MAX_B;
  const size_t places = static_cast<size_t>(l.slots) * 2 * heads;
  l.tags = (static_cast<size_t>(pages) * 2 * heads * sizeof(uint32_t) + 255) / 256 * 256;
  l.codes = l.tags + (places * sizeof(KeptTag) + 255) / 256 * 256;
  l.total = l.codes + places * DG_PAGE * dim;
  return l;
}

// Two sums over the block's threads.
DG_DEV uint2 block_check(uint32_t a, uint32_t b, uint32_t* sums /* [2][threads / 32] shared */) {
  const int warps = blockDim.x >> 5;
  a = __reduce_add_sync(0xffffffffu, a);
  b = __reduce_add_sync(0xffffffffu, b);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    sums[threadIdx.x >> 5] = a;
    sums[warps + (threadIdx.x >> 5)] = b;
  }
  __syncthreads();
  uint2 t = make_uint2(0, 0);
  for (int w = 0; w < warps; ++w) {
    t.x += sums[w];
    t.y += sums[warps + w];
  }
  return t;
}
DG_DEV void check_word(uint32_t i, uint32_t w, uint32_t& a, uint32_t& b) {
  uint32_t x = (w + i * 0x9E3779B9u) * 0x85EBCA6Bu;
  x ^= x >> 15;
  a += x * 0xC2B2AE35u;
  b += (x ^ (x >> 13)) * 0x27D4EB2Fu;
}

constexpr int kMine = 2;
constexpr int kAppendHeads = 128;  // heads of a block at most
template <int kDim>
constexpr int kAppendThreads = DG_PAGE * kDim / 16 / kMine;
static_assert(kAppendThreads<64> >= kAppendHeads, "a thread for each head's mark");

// The tags and the codes put aside of a run's heads, from head 0 on; tags null:
// nothing is put aside.  All threads of the block.
struct KeptPlace {
  KeptTag* tags;
  uint32_t* codes;
  uint32_t epoch;
};
template <int kDim>
DG_DEV KeptPlace kept_place(const dg_context& c, const dg_context_cache& cache, bool is_k, int page, int row0, uint32_t* sums) {
  KeptPlace k = {nullptr, nullptr, 0};
  if (cache.kept == nullptr || c.epoch == nullptr) return k;
  int slot = page;
  if (cache.pages > DG_MAX_B) {  // the request whose first row this is
    uint32_t r = 0;
    for (int i = threadIdx.x; i < c.B; i += blockDim.x) {
      if (c.start[i] == row0 && c.start[i + 1] > row0) r = i + 1;
    }
    slot = static_cast<int>(block_check(r, 0, sums).x) - 1;
    if (slot < 0 || slot >= DG_MAX_B) return k;
  }
  const KeptLayout l = kept_layout(cache.pages, cache.heads, kDim);
  const size_t at = (static_cast<size_t>(slot) * 2 + (is_k ? 0 : 1)) * cache.heads;
  k.tags = reinterpret_cast<KeptTag*>(cache.kept + l.tags) + at;
  k.codes = reinterpret_cast<uint32_t*>(cache.kept + l.codes + at * DG_PAGE * kDim);
  k.epoch = static_cast<uint32_t>(*c.epoch);
  return k;
}

// One head of a run behind held tokens whose scale the new rows want to be `s`,
// where that is above the page's, or where the page's has grown before: the
// held codes under the scale that comes of it, that scale, and the rows' codes.
// By a block, or (kBlock false) by a warp.
template <int kDim, bool kBlock>
DG_DEV void append_grown_head(const dg_context_cache& cache, const dg_heads& in, uint32_t* marks,
                              const float2 (*turns)[kDim / 2], int rot16, bool il, bool is_k, int4 run, int h, float s,
                              const KeptPlace& k, uint32_t* sums) {
  constexpr int kUnits = kDim / 16, kTeam = kBlock ? kAppendThreads<kDim> : 32;
  constexpr int kAtOnce = 8;  // words on their way: all that a block has of a page
  const int t = kBlock ? threadIdx.x : (threadIdx.x & 31);
  const int page = run.x, row0 = run.y, off = run.z, n = run.w;
  const size_t at = static_cast<size_t>(page) * cache.heads + h;
  uint8_t* page_codes = (is_k ? cache.k : cache.v) + at * DG_PAGE * kDim;
  uint32_t* codes = reinterpret_cast<uint32_t*>(page_codes);
  float* scale = (is_k ? cache.k_scale : cache.v_scale) + at;
  KeptTag* tag = k.tags == nullptr ? nullptr : k.tags + h;
  uint32_t* kept = k.codes + static_cast<size_t>(h) * (DG_PAGE * kDim / 4);
  const int words = off * kDim / 4;
  auto check = [&](uint32_t a, uint32_t b) {  // over the team, every thread past what it read before
    if (kBlock) return block_check(a, b, sums);
    return make_uint2(__reduce_add_sync(0xffffffffu, a), __reduce_add_sync(0xffffffffu, b));
  };
  const float old = *scale;
  bool mine = false, restore = false;  // the tag is of this page as it stands: of this plan's batch, or of another's
  float base = old;
  uint32_t a = 0, b = 0;
  if (tag != nullptr && tag->page == page && tag->off == off && __float_as_uint(tag->grown) == __float_as_uint(old) &&
      marks[at] == grown_mark(tag->epoch, off)) {
    for (int i0 = t; i0 < words; i0 += kAtOnce * kTeam) {
      uint32_t w[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) w[j] = i0 + j * kTeam < words ? codes[i0 + j * kTeam] : 0u;
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        if (i0 + j * kTeam < words) check_word(i0 + j * kTeam, w[j], a, b);
      }
    }
    const uint2 sum = check(a, b);
    const bool same = sum.x == tag->check[0] && sum.y == tag->check[1];
    mine = same && tag->epoch == k.epoch;
    restore = same && !mine;
    if (restore) base = tag->base;
  }
  const bool grows = s > base;
  if (!grows) s = base;
  a = b = 0;
  if (grows || restore) {
    const float ratio = base / s;
    const uint32_t* from = restore ? kept : codes;
    for (int i0 = t; i0 < words; i0 += kAtOnce * kTeam) {
      uint32_t w[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) w[j] = i0 + j * kTeam < words ? from[i0 + j * kTeam] : 0u;
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int i = i0 + j * kTeam;
        if (i >= words) continue;
        if (grows) {
          if (tag != nullptr && !mine && !restore) kept[i] = w[j];
          float f[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __half_raw hr = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(w[j] >> (8 * e)), __NV_E4M3);
            f[e] = __half2float(*reinterpret_cast<const __half*>(&hr)) * ratio;
          }
          w[j] = e4m3_pair(f[0], f[1]) | e4m3_pair(f[2], f[3]) << 16;
        }
        codes[i] = w[j];
        check_word(i, w[j], a, b);
      }
    }
  }
  const uint2 sum = check(a, b);
  if (t == 0) {
    *scale = s;
    if (tag != nullptr && grows) {
      if (!mine) {
        tag->page = page;
        tag->off = off;
        tag->epoch = k.epoch;
        tag->base = base;
      }
      tag->grown = s;
      tag->check[0] = sum.x;
      tag->check[1] = sum.y;
      marks[at] = grown_mark(k.epoch, off);
    } else if (tag != nullptr) {  // as it was, or written by somebody else
      tag->off = 0;
      marks[at] = 0;
    }
  }
  const float inv = 1.0f / s;  // exact: a power of two
  const int u = t % kUnits;
  int ca, cb;
  unit_chunks(u, rot16, il, ca, cb);
  constexpr int kRows = kTeam / kUnits;
  const uint8_t* src = static_cast<const uint8_t*>(in.data) + 2 * h * in.head_stride;
  for (int r0 = t / kUnits; r0 < n; r0 += kMine * kRows) {
    uint4 wa[kMine], wb[kMine];
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      const uint8_t* row = src + 2 * (row0 + min(r0 + m * kRows, n - 1)) * in.row_stride;
      wa[m] = *reinterpret_cast<const uint4*>(row + 16 * ca);
      wb[m] = *reinterpret_cast<const uint4*>(row + 16 * cb);
    }
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      const int row = r0 + m * kRows;
      if (row >= n) continue;
      float x[8], y[8];
      unpack8(wa[m], x);
      unpack8(wb[m], y);
      if (u < rot16) {
        float2 tr[8];
        read_turns(turns[row], u, rot16, tr);
        rotate_unit(x, y, tr, il);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {  // NaN becomes 0
        if (x[j] != x[j]) x[j] = 0.f;
        if (y[j] != y[j]) y[j] = 0.f;
      }
      uint8_t* dst = page_codes + (off + row) * kDim;
      *reinterpret_cast<uint2*>(dst + 8 * ca) = e4m3_chunk(x, inv);
      *reinterpret_cast<uint2*>(dst + 8 * cb) = e4m3_chunk(y, inv);
    }
  }
}

// The heads of a list, each with the scale that its rows want.  All threads of
// the block: a head after the other, or, of many, a warp to each.  Out of line
// and on its own: within the loop over the heads its registers cost every append
// (256 requests x 8 heads x 1 row 12.9 us instead of 12.4).
struct GrownHead {
  int head;
  float want;
};
template <int kDim>
__device__ __noinline__ void append_grown(const dg_context& c, const dg_context_cache& cache, const dg_heads& in,
                                          const float2 (*turns)[kDim / 2], int rot16, bool il, bool is_k, int4 run,
                                          const GrownHead* list, int count, uint32_t* sums) {
  const KeptPlace k = kept_place<kDim>(c, cache, is_k, run.x, run.y, sums);
  uint32_t* marks = kept_marks(cache, is_k);
  if (count <= 2) {
    for (int i = 0; i < count; ++i)
      append_grown_head<kDim, true>(cache, in, marks, turns, rot16, il, is_k, run, list[i].head, list[i].want, k, sums);
  } else {
    for (int i = threadIdx.x >> 5; i < count; i += blockDim.x >> 5)
      append_grown_head<kDim, false>(cache, in, marks, turns, rot16, il, is_k, run, list[i].head, list[i].want, k, sums);
  }
}

// One CTA per (run, `per` kv heads, k or v): it owns those pages' scales and
// all of their codes, so no two CTAs meet.  A thread has kMine units of 16
// elements (a run of 64 rows fills the block); they stay in registers between
// the two things that need them, the largest magnitude and the codes, and the
// next head's are on their way meanwhile.  The turns of the run's tokens are
// formed once and serve all of its heads.
// Measured (8 heads x 128): 32 requests x 256 rows, 50 MB, in 17.9 us from HBM,
// 2.8 TB/s, and 12.4 one after another with the rows in L2; bound by latency at
// two blocks an SM (105 registers a thread; squeezed to 78 and 64 for three and
// four blocks it took 17.6 and 23.5 us where two took 12.3, in L2); 32 requests x
// 1 row in 3.5 us.  Behind a plan that had another batch raise every scale of
// its pages, 32 x 256 rows take 22 us, 32 x 1 row 11.
template <int kDim>
__global__ void __launch_bounds__(kAppendThreads<kDim>)
context_append_kernel(const __grid_constant__ dg_context c, const __grid_constant__ dg_context_cache cache,
                      const __grid_constant__ dg_heads kin, const __grid_constant__ dg_heads vin, const dg_rope_args rope,
                      int has_rope, int per) {
  constexpr int kUnits = kDim / 16;  // units per row
  constexpr int kThreads = kAppendThreads<kDim>, kWarps = kThreads / 32;
  constexpr int kRows = kThreads / kUnits;        // rows between a thread's units
  __shared__ float s_top[3][kWarps];
  __shared__ __align__(16) float2 s_turn[DG_PAGE][kDim / 2];
  __shared__ uint32_t s_check[2 * kWarps];
  __shared__ uint32_t s_bits[kAppendHeads / 32];
  __shared__ GrownHead s_grown[kAppendHeads];
  wait_for_previous_kernel();
  allow_next_kernel();
  const int4 run = reinterpret_cast<const int4*>(c.runs)[blockIdx.x];
  const int page = run.x, row0 = run.y, off = run.z, n = run.w;
  if (page < 0 || page >= cache.pages || n <= 0 || off < 0 || off + n > DG_PAGE || row0 < 0 || row0 + n > c.rows) return;
  const int head0 = blockIdx.y * per, heads = min(per, cache.heads - head0);
  const bool is_k = blockIdx.z == 0;
  const dg_heads& in = is_k ? kin : vin;
  const int rot16 = (is_k && has_rope) ? rope.rot / 16 : 0;
  const bool il = rope.interleaved != 0;
  const int row = threadIdx.x / kUnits, u = threadIdx.x % kUnits;  // of the thread's first unit
  const bool turned = u < rot16;
  int ca, cb;
  unit_chunks(u, rot16, il, ca, cb);
  const size_t at0 = static_cast<size_t>(page) * cache.heads + head0;
  float* scale = (is_k ? cache.k_scale : cache.v_scale) + at0;
  uint8_t* codes = (is_k ? cache.k : cache.v) + at0 * DG_PAGE * kDim;
  const uint8_t* src = static_cast<const uint8_t*>(in.data) + 2 * ((row0 + row) * in.row_stride + head0 * in.head_stride);
  const int64_t row_step = 2 * kRows * in.row_stride, head_step = 2 * in.head_stride;

  uint4 wa[kMine] = {}, wb[kMine] = {};
  auto load = [&](const uint8_t* from) {
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      if (row + m * kRows >= n) continue;
      wa[m] = *reinterpret_cast<const uint4*>(from + m * row_step + 16 * ca);
      wb[m] = *reinterpret_cast<const uint4*>(from + m * row_step + 16 * cb);
    }
  };
  load(src);
  // Heads whose scale another plan's batch behind the same tokens has made to
  // grow.  A page that is begun has not grown.
  bool grown = false;
  if (static_cast<int>(threadIdx.x) < heads && cache.kept != nullptr && c.epoch != nullptr) {
    uint32_t* mark = kept_marks(cache, is_k) + at0 + threadIdx.x;
    if (off > 0) {
      const uint32_t m = *mark, now = grown_mark(static_cast<uint32_t>(*c.epoch), off);
      grown = m != now && (m & (DG_PAGE - 1)) == (now & (DG_PAGE - 1));
    } else {
      *mark = 0;
    }
  }
  int later = 0;  // heads for append_grown
  if (rot16 > 0) {
    const int half = 8 * rot16, stride = kThreads / half;
    const int j = threadIdx.x % half;  // this thread's frequency; the block's threads walk the rows
    const uint64_t turn = turn_fraction(rope.freq[j]);
    const uint32_t pos = c.positions[row0];  // a run's tokens follow one another
    for (int r = threadIdx.x / half; r < n && static_cast<int>(threadIdx.x) < stride * half; r += stride)
      s_turn[r][turn_place(j, rot16)] = turn_of((pos + r) * turn, rope.magnitude);
    __syncthreads();
  }
  for (int h = 0; h < heads; ++h, ++scale, codes += DG_PAGE * kDim) {
    const float old = *scale;
    float a[kMine][8], b[kMine][8];
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      unpack8(wa[m], a[m]);
      unpack8(wb[m], b[m]);
    }
    src += head_step;
    if (h + 1 < heads) load(src);
    if (turned) {
#pragma unroll
      for (int m = 0; m < kMine; ++m) {
        if (row + m * kRows >= n) continue;
        float2 tr[8];
        read_turns(s_turn[row + m * kRows], u, rot16, tr);
        rotate_unit(a[m], b[m], tr, il);
      }
    }
    float top = 0.f, zero = 0.f, zero2 = 0.f;  // sums of 0 x: NaN if some x is not finite
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        top = fmaxf(top, fmaxf(fabsf(a[m][j]), fabsf(b[m][j])));
        zero = fmaf(a[m][j], 0.f, zero);
        zero2 = fmaf(b[m][j], 0.f, zero2);
      }
    }
    zero += zero2;
    // The largest over the block; infinite if anything is not finite.  The
    // barrier also has every thread past its read of the old scale.
    auto largest = [&](int buffer) {
      top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));  // not negative: ordered as integers
      if ((threadIdx.x & 31) == 0) s_top[buffer][threadIdx.x >> 5] = top;
      __syncthreads();
      top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(s_top[buffer][threadIdx.x & (kWarps - 1)])));
    };
    if (zero != zero) top = INFINITY;
    if (h == 0 && threadIdx.x < kAppendHeads) {
      const uint32_t bits = __ballot_sync(0xffffffffu, grown);
      if ((threadIdx.x & 31) == 0) s_bits[threadIdx.x >> 5] = bits;
    }
    largest(h & 1);
    if (top > FLT_MAX) {  // seldom: what is not finite does not count, NaN becomes 0
      top = 0.f;
#pragma unroll
      for (int m = 0; m < kMine; ++m) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x = fabsf(a[m][j]), y = fabsf(b[m][j]);
          if (x <= FLT_MAX) top = fmaxf(top, x);
          if (y <= FLT_MAX) top = fmaxf(top, y);
          if (a[m][j] != a[m][j]) a[m][j] = 0.f;
          if (b[m][j] != b[m][j]) b[m][j] = 0.f;
        }
      }
      largest(2);
      if (threadIdx.x == 0) atomicOr(reinterpret_cast<unsigned*>(c.status + 1), 1u);
      __syncthreads();  // the third buffer may be used again
    }
    const int e = scale_exponent(top);
    float s = power_of_two(e), inv = power_of_two(-e);  // |e| <= 120
    if (off > 0) {
      if (s > old || (s_bits[h >> 5] >> (h & 31) & 1u)) {
        if (threadIdx.x == 0) s_grown[later] = GrownHead{head0 + h, s};
        ++later;
        continue;
      }
      s = old;
      inv = 1.0f / old;  // exact: a power of two
    }
    uint8_t* dst = codes + (off + row) * kDim;
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      if (row + m * kRows >= n) continue;
      *reinterpret_cast<uint2*>(dst + m * kRows * kDim + 8 * ca) = e4m3_chunk(a[m], inv);
      *reinterpret_cast<uint2*>(dst + m * kRows * kDim + 8 * cb) = e4m3_chunk(b[m], inv);
    }
    if (threadIdx.x == 0) *scale = s;
  }
  if (later > 0) {
    __syncthreads();
    append_grown<kDim>(c, cache, in, s_turn, rot16, il, is_k, run, s_grown, later, s_check);
  }
}

bool aligned(const void* p, uintptr_t n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

dg_status check_rope(const dg_rope_args* r, int dim) {
  if (r->rot < 16 || r->rot % 16 != 0 || r->rot > dim || !aligned(r->freq, 8)) return DG_ERR_INVALID_ARG;
  if (!(fabsf(r->magnitude) <= 3.0e38f)) return DG_ERR_INVALID_ARG;
  return DG_OK;
}

}  // namespace

dg_status check_context(const dg_context* c) {
  if (c == nullptr) return DG_ERR_INVALID_ARG;
  if (c->B < 1 || c->B > DG_MAX_B || c->rows < 1 || c->rows > kContextMaxRows || c->pages < 1 ||
      c->pages > (1 << 24) || c->max_pages < 1 || c->max_pages > (1 << 24))
    return DG_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(c->table, 4) || !aligned(c->held, 4) || !aligned(c->free_list, 4) || !aligned(c->free_count, 4) ||
      !aligned(c->lens, 4) || !aligned(c->start, 4) || !aligned(c->positions, 4) || !aligned(c->slots, 8) ||
      !aligned(c->runs, 16) || !aligned(c->free_next, 4) || !aligned(c->status, 4) ||
      (c->epoch != nullptr && !aligned(c->epoch, 4)))
    return DG_ERR_INVALID_ARG;
  return DG_OK;
}

dg_status check_heads(const dg_heads* t, int heads, int dim) {
  if (t == nullptr || !aligned(t->data, 16)) return DG_ERR_INVALID_ARG;
  if (t->row_stride % 8 != 0 || t->head_stride % 8 != 0) return DG_ERR_INVALID_ARG;
  if (t->row_stride < dim || t->row_stride > (int64_t(1) << 40) || t->head_stride > (int64_t(1) << 40) ||
      (heads > 1 && t->head_stride < dim))
    return DG_ERR_INVALID_ARG;
  return DG_OK;
}

dg_status check_cache(const dg_context_cache* c, const dg_context* ctx) {
  if (c == nullptr) return DG_ERR_INVALID_ARG;
  if ((c->dim != 64 && c->dim != 128) || c->heads < 1 || c->heads > 1024 || c->pages != ctx->pages)
    return DG_ERR_UNSUPPORTED_SHAPE;
  if (static_cast<int64_t>(c->pages) * c->heads * DG_PAGE > 0x7fffffffll - 1025 * DG_PAGE) return DG_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
      (c->kept != nullptr && !aligned(c->kept, 16)))
    return DG_ERR_INVALID_ARG;
  return DG_OK;
}

}  // namespace dg

using namespace dg;

extern "C" {

dg_status dg_context_plan(const dg_context* ctx, const int32_t* add, const uint8_t* release, int32_t commit,
                          void* stream) {
  const dg_status st = check_context(ctx);
  if (st != DG_OK) return st;
  if (!aligned(add, 4)) return DG_ERR_INVALID_ARG;
  if (device_sms() <= 0) return DG_ERR_NO_DEVICE;
  return cuda_ok(launch_context(context_plan_kernel, dim3(kPlanCtas), kPlanThreads, 0, static_cast<cudaStream_t>(stream),
                                *ctx, add, release, commit),
                 "context plan launch")
             ? DG_OK
             : DG_ERR_CUDA;
}

dg_status dg_context_status(const dg_context* ctx, void* stream) {
  const dg_status ck = check_context(ctx);
  if (ck != DG_OK) return ck;
  if (device_sms() <= 0) return DG_ERR_NO_DEVICE;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  int32_t s[2] = {0, 0};
  if (!cuda_ok(cudaMemcpyAsync(s, ctx->status, sizeof(s), cudaMemcpyDeviceToHost, cs), "context status read") ||
      !cuda_ok(cudaStreamSynchronize(cs), "stream synchronise"))
    return DG_ERR_CUDA;
  if (s[0] != 0) {
    set_last_error_message(s[0] == 1   ? "the context's pool has too few free pages for the batch"
                           : s[0] == 2 ? "the batch has more rows than the context"
                                       : "a length is negative or beyond the context's table");
    return DG_ERR_CAPACITY;
  }
  if (s[1] != 0) {  // reported, so it may go
    if (!cuda_ok(cudaMemsetAsync(ctx->status + 1, 0, sizeof(int32_t), cs), "context latch clear")) return DG_ERR_CUDA;
    set_last_error_message("a key or value appended to the context is not finite");
    return DG_ERR_VALUE;
  }
  return DG_OK;
}

dg_status dg_rope_frequencies(int32_t rot, double base, int32_t scaling, double factor, int32_t original_length,
                              double* freq, float* magnitude) {
  if (rot < 16 || rot % 16 != 0 || rot > 128) return DG_ERR_UNSUPPORTED_SHAPE;
  if (freq == nullptr || magnitude == nullptr || !(base > 1.0 && base < 1e300) || !(factor >= 1.0 && factor < 1e9) ||
      scaling < DG_ROPE_NONE || scaling > DG_ROPE_PARTS || original_length < 1)
    return DG_ERR_INVALID_ARG;
  if (scaling == DG_ROPE_NTK) base *= pow(factor, static_cast<double>(rot) / (rot - 2));
  // The pair index at which a pair makes `turns` turns over original_length
  // positions; the ramp of PARTS lies between those of 32 turns and 1 turn.
  auto pair_at = [&](double turns) {
    return rot * log(original_length / (turns * 6.283185307179586)) / (2.0 * log(base));
  };
  const double low = fmax(floor(pair_at(32.0)), 0.0), high = fmin(ceil(pair_at(1.0)), rot - 1.0);
  const double width = fmax(high - low, 1e-3);
  for (int j = 0; j < rot / 2; ++j) {
    double f = pow(base, -2.0 * j / rot);
    if (scaling == DG_ROPE_LINEAR) f /= factor;
    if (scaling == DG_ROPE_PARTS) {
      const double ramp = fmin(fmax((j - low) / width, 0.0), 1.0);
      f = f / factor * ramp + f * (1.0 - ramp);
    }
    freq[j] = f;
  }
  *magnitude = scaling == DG_ROPE_PARTS ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.0f;
  return DG_OK;
}

dg_status dg_rope(const dg_heads* x, const dg_heads* out, int32_t rows, int32_t heads, int32_t dim,
                  const int32_t* positions, const dg_rope_args* rope, void* stream) {
  if (rows < 0 || rows > kContextMaxRows || heads < 1 || heads > 65536 || (dim != 64 && dim != 128))
    return DG_ERR_UNSUPPORTED_SHAPE;
  dg_status st;
  if ((st = check_heads(x, heads, dim)) != DG_OK || (st = check_heads(out, heads, dim)) != DG_OK) return st;
  if (x->data == out->data && (x->row_stride != out->row_stride || x->head_stride != out->head_stride))
    return DG_ERR_INVALID_ARG;
  if (!aligned(positions, 4) || rope == nullptr) return DG_ERR_INVALID_ARG;
  if ((st = check_rope(rope, dim)) != DG_OK) return st;
  const int sms = device_sms();
  if (sms <= 0) return DG_ERR_NO_DEVICE;
  if (rows == 0) return DG_OK;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const int stride = kRopeThreads / (dim / 16);
  auto launch = [&](auto kernel, int tokens) {
    return launch_context(kernel, dim3((rows + tokens - 1) / tokens), kRopeThreads, 0, cs,
                          static_cast<const uint8_t*>(x->data), static_cast<uint8_t*>(out->data), x->row_stride,
                          x->head_stride, out->row_stride, out->head_stride, rows, heads, stride / heads,
                          stride % heads, positions, rope->freq, rope->rot, rope->interleaved, rope->magnitude);
  };
  // Few rows: a CTA per row, for the latency; more: four or eight, for fewer
  // starts and a longer stream per thread, 32 where a row is short.  In us, 22
  // heads x 128 with 1 / 4 rows a CTA: 32 rows 1.9 / 2.5, 592 rows 2.5 / 2.7,
  // 1184 rows 4.2 / 3.2.  With 4 / 8 (inputs from HBM): 2000 x 22 heads 5.2 / 5.7,
  // 4000 x 16 8.2 / 7.6, 8191 x 16 14.2 / 13.1, 8191 x 32 23.3 / 23.9.  With 8 / 32:
  // 16384 x 8 14.8 / 15.7, 32768 x 4 18.7 / 17.0, 131072 x 1 60 / 39.
  const int64_t width = static_cast<int64_t>(heads) * dim;
  const int tokens = rows <= 4 * sms ? 1 : (rows < 24 * sms || width >= 4096) ? 4 : width > 512 ? 8 : 32;
  auto start = [&](auto one, auto four, auto eight, auto many) {
    return tokens == 1 ? launch(one, 1) : tokens == 4 ? launch(four, 4) : tokens == 8 ? launch(eight, 8) : launch(many, 32);
  };
  const cudaError_t e =
      dim == 128 ? start(rope_kernel<128, 1>, rope_kernel<128, 4>, rope_kernel<128, 8>, rope_kernel<128, 32>)
                 : start(rope_kernel<64, 1>, rope_kernel<64, 4>, rope_kernel<64, 8>, rope_kernel<64, 32>);
  return cuda_ok(e, "rope launch") ? DG_OK : DG_ERR_CUDA;
}

size_t dg_context_kept_size(int32_t pages, int32_t heads, int32_t dim) {
  if (pages < 1 || pages > (1 << 24) || heads < 1 || heads > 1024 || (dim != 64 && dim != 128)) return 0;
  return kept_layout(pages, heads, dim).total;
}

dg_status dg_context_append(const dg_context* ctx, const dg_context_cache* cache, const dg_heads* k,
                            const dg_heads* v, const dg_rope_args* rope, void* stream) {
  dg_status st;
  if ((st = check_context(ctx)) != DG_OK || (st = check_cache(cache, ctx)) != DG_OK) return st;
  if ((st = check_heads(k, cache->heads, cache->dim)) != DG_OK) return st;
  if ((st = check_heads(v, cache->heads, cache->dim)) != DG_OK) return st;
  if (rope != nullptr && (st = check_rope(rope, cache->dim)) != DG_OK) return st;
  const int sms = device_sms();
  if (sms <= 0) return DG_ERR_NO_DEVICE;
  const dg_rope_args none = {};
  // More heads a CTA save turns and starts, until too few CTAs are left to
  // fill the device: up to 3.5 an SM.  1 / 2 / 4 / 8 heads a CTA, in us (8 heads
  // x 128, one after another): 32 requests x 1 row 4.5 / 3.6 / 4.4 / 5.7; 4 x 256
  // rows 4.2 / 5.1 / 6.0 / 7.9; 16 x 256 12.3 / 9.7 / 8.0 / 11.2; 32 x 256 20.9 /
  // 15.3 / 13.0 / 11.9.
  const int runs = DG_CONTEXT_RUNS(ctx->rows, ctx->B);
  int per = 1;
  while (per < cache->heads && per < kAppendHeads && 4ll * runs * ((cache->heads + per - 1) / per) > 7ll * sms) per *= 2;
  const dim3 grid(runs, (cache->heads + per - 1) / per, 2);
  auto kernel = cache->dim == 128 ? context_append_kernel<128> : context_append_kernel<64>;
  const cudaError_t e = launch_context(kernel, grid, cache->dim * (DG_PAGE / 16) / kMine, 0, static_cast<cudaStream_t>(stream),
                                       *ctx, *cache, *k, *v, rope ? *rope : none, rope != nullptr, per);
  return cuda_ok(e, "context append launch") ? DG_OK : DG_ERR_CUDA;
}

}  // extern "C"
