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
// in hardware instead of three launches in a row.
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
  for (int i = gtid; i < c.rows; i += gsize) {
    int pos = -1;
    int64_t slot = -1;
    if (i < total) {
      const int r = owner_of(s_start, B, i);
      pos = s_held[r] + i - s_start[r];
      slot = static_cast<int64_t>(page_of(r, pos / DG_PAGE)) * DG_PAGE + pos % DG_PAGE;
    }
    c.positions[i] = pos;
    c.slots[i] = slot;
  }
  const int runs = DG_CONTEXT_RUNS(c.rows, B), used = s_run0[B];
  for (int u = gtid; u < runs; u += gsize) {
    int4 run = make_int4(-1, 0, 0, 0);
    if (u < used) {
      const int r = owner_of(s_run0, B, u);
      const int h = s_held[r], end = h + s_start[r + 1] - s_start[r];
      const int j = h / DG_PAGE + u - s_run0[r];
      const int lo = max(j * DG_PAGE, h), hi = min((j + 1) * DG_PAGE, end);
      run = make_int4(page_of(r, j), s_start[r] + lo - h, lo - j * DG_PAGE, hi - lo);
    }
    reinterpret_cast<int4*>(c.runs)[u] = run;
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
// cos and sin of position * freq, times the magnitude.  The product and its
// reduction to a fraction of a turn are in float64 (a float32 product is off
// by more than a hundredth of a radian at positions in the hundred
// thousands); the fraction, at most half a turn, is then exact enough in
// float32 for sincospif.
DG_DEV float2 turn_of(int position, double freq, float magnitude) {
  double t = static_cast<double>(position) * freq * 0.15915494309189533577;  // 1 / (2 pi)
  t -= rint(t);
  float s, c;
  sincospif(2.0f * static_cast<float>(t), &s, &c);
  return make_float2(c * magnitude, s * magnitude);
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
DG_DEV void rotate_unit(float (&a)[8], float (&b)[8], const float2 (&t)[8], bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = a[2 * i], y = a[2 * i + 1];
      a[2 * i] = x * t[i].x - y * t[i].y;
      a[2 * i + 1] = x * t[i].y + y * t[i].x;
      const float z = b[2 * i], w = b[2 * i + 1];
      b[2 * i] = z * t[4 + i].x - w * t[4 + i].y;
      b[2 * i + 1] = z * t[4 + i].y + w * t[4 + i].x;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = a[i], y = b[i];
      a[i] = x * t[i].x - y * t[i].y;
      b[i] = x * t[i].y + y * t[i].x;
    }
  }
}

constexpr int kRopeThreads = 256;

// kTokens token rows per CTA.  The turns of a token serve all of its heads:
// they are formed once, by one thread per (token, frequency), and kept in
// shared memory; the heads then stream through, 32 bytes a thread.
template <int kTokens>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(const uint8_t* x, uint8_t* out, int64_t xr, int64_t xh, int64_t outr, int64_t outh, int rows,
            int heads, int dim, const int32_t* __restrict__ positions, const double* __restrict__ freq, int rot,
            int interleaved, float magnitude) {
  __shared__ float2 turns[kTokens][64];
  __shared__ int s_pos[kTokens];
  const int row0 = blockIdx.x * kTokens;
  const int half = rot / 2;
  for (int i = threadIdx.x; i < kTokens * half; i += kRopeThreads) {
    const int t = i / half, j = i - t * half;
    if (row0 + t < rows) turns[t][j] = turn_of(positions[row0 + t], freq[j], magnitude);
  }
  if (threadIdx.x < kTokens) s_pos[threadIdx.x] = row0 + threadIdx.x < rows ? positions[row0 + threadIdx.x] : -1;
  __syncthreads();
  const int units = dim / 16, rot16 = rot / 16;
  const int per_token = heads * units;
  const bool in_place = x == out;
  for (int i = threadIdx.x; i < kTokens * per_token; i += kRopeThreads) {
    const int t = i / per_token, rest = i - t * per_token;
    const int h = rest / units, u = rest - h * units;
    if (s_pos[t] < 0 || (in_place && u >= rot16)) continue;
    int ca, cb;
    unit_chunks(u, rot16, interleaved, ca, cb);
    const uint8_t* src = x + 2 * ((row0 + t) * xr + h * xh);
    uint8_t* dst = out + 2 * ((row0 + t) * outr + h * outh);
    uint4 wa = *reinterpret_cast<const uint4*>(src + 16 * ca), wb = *reinterpret_cast<const uint4*>(src + 16 * cb);
    if (u < rot16) {
      float a[8], b[8];
      unpack8(wa, a);
      unpack8(wb, b);
      float2 tr[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) tr[j] = turns[t][8 * u + j];
      rotate_unit(a, b, tr, interleaved);
      wa = pack8(a);
      wb = pack8(b);
    }
    *reinterpret_cast<uint4*>(dst + 16 * ca) = wa;
    *reinterpret_cast<uint4*>(dst + 16 * cb) = wb;
  }
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 256;

// The least power of two s with top <= 448 s, at least 2^-100; 1 for 0.
// 448 = 0.875 * 2^9, so with top = f 2^e (f in [0.5, 1)) s is 2^(e - 9) for
// f <= 0.875 and 2^(e - 8) above.
DG_DEV float scale_of(float top) {
  if (top == 0.f) return 1.f;
  int e;
  const float f = frexpf(top, &e);
  e = max(e - 9 + (f > 0.875f ? 1 : 0), -100);
  return ldexpf(1.f, e);
}
// Two floats to E4M3, to nearest even, saturating; NaN stays NaN.
DG_DEV uint32_t e4m3_pair(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
DG_DEV uint2 e4m3_chunk(const float (&x)[8], float inv) {
  return make_uint2(e4m3_pair(x[0] * inv, x[1] * inv) | e4m3_pair(x[2] * inv, x[3] * inv) << 16,
                    e4m3_pair(x[4] * inv, x[5] * inv) | e4m3_pair(x[6] * inv, x[7] * inv) << 16);
}

// One CTA per (run, kv head, k or v): it owns the page's scale and all of
// its codes, so no two CTAs meet.  The run's values stay in registers
// between the two things that need them, the largest magnitude and the
// codes: 64 rows x 128 elements are 32 floats a thread.
template <int kDim>
__global__ void __launch_bounds__(kAppendThreads)
context_append_kernel(const dg_context c, const dg_context_cache cache, const dg_heads kin, const dg_heads vin,
                      const dg_rope_args rope, int has_rope) {
  constexpr int kUnits = kDim / 16;                                  // units per row
  constexpr int kMine = DG_PAGE * kUnits / kAppendThreads;           // units per thread
  __shared__ float s_top[kAppendThreads / 32];
  const int4 run = reinterpret_cast<const int4*>(c.runs)[blockIdx.x];
  const int page = run.x, row0 = run.y, off = run.z, n = run.w;
  if (page < 0 || page >= cache.pages || n <= 0 || off < 0 || off + n > DG_PAGE || row0 < 0 || row0 + n > c.rows) return;
  const int head = blockIdx.y;
  const bool is_k = blockIdx.z == 0;
  const dg_heads& in = is_k ? kin : vin;
  float* scale_at = (is_k ? cache.k_scale : cache.v_scale) + static_cast<size_t>(page) * cache.heads + head;
  uint8_t* codes = (is_k ? cache.k : cache.v) + (static_cast<size_t>(page) * cache.heads + head) * DG_PAGE * kDim;
  const int rot16 = (is_k && has_rope) ? rope.rot / 16 : 0;
  const bool il = rope.interleaved != 0;

  float a[kMine][8], b[kMine][8];
  float top = 0.f;
  bool odd = false;
#pragma unroll
  for (int m = 0; m < kMine; ++m) {
    const int i = threadIdx.x + m * kAppendThreads;
    const int row = i / kUnits, u = i % kUnits;
    if (row >= n) continue;
    int ca, cb;
    unit_chunks(u, rot16, il, ca, cb);
    const uint8_t* src = static_cast<const uint8_t*>(in.data) + 2 * ((row0 + row) * in.row_stride + head * in.head_stride);
    unpack8(*reinterpret_cast<const uint4*>(src + 16 * ca), a[m]);
    unpack8(*reinterpret_cast<const uint4*>(src + 16 * cb), b[m]);
    if (u < rot16) {
      const int pos = c.positions[row0 + row];
      float2 tr[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) tr[j] = turn_of(pos, rope.freq[8 * u + j], rope.magnitude);
      rotate_unit(a[m], b[m], tr, il);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = fabsf(a[m][j]), y = fabsf(b[m][j]);
      if (x <= FLT_MAX) top = fmaxf(top, x); else odd = true;
      if (y <= FLT_MAX) top = fmaxf(top, y); else odd = true;
      if (a[m][j] != a[m][j]) a[m][j] = 0.f;
      if (b[m][j] != b[m][j]) b[m][j] = 0.f;
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
  if (__any_sync(0xffffffffu, odd) && (threadIdx.x & 31) == 0) atomicOr(reinterpret_cast<unsigned*>(c.status + 1), 1u);
  const float old = *scale_at;
  __syncthreads();
  top = s_top[0];
#pragma unroll
  for (int w = 1; w < kAppendThreads / 32; ++w) top = fmaxf(top, s_top[w]);
  float s = scale_of(top);
  if (off > 0 && !(s > old)) s = old;
  if (off > 0 && s > old) {  // kept tokens move to the larger scale
    const float ratio = old / s;
    for (int i = threadIdx.x; i < off * kDim / 4; i += kAppendThreads) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(codes)[i];
      float f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half_raw hr = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(w >> (8 * j)), __NV_E4M3);
        f[j] = __half2float(*reinterpret_cast<const __half*>(&hr)) * ratio;
      }
      reinterpret_cast<uint32_t*>(codes)[i] = e4m3_pair(f[0], f[1]) | e4m3_pair(f[2], f[3]) << 16;
    }
  }
  const float inv = 1.0f / s;  // exact: s is a power of two
#pragma unroll
  for (int m = 0; m < kMine; ++m) {
    const int i = threadIdx.x + m * kAppendThreads;
    const int row = i / kUnits, u = i % kUnits;
    if (row >= n) continue;
    int ca, cb;
    unit_chunks(u, rot16, il, ca, cb);
    uint8_t* dst = codes + (off + row) * kDim;
    *reinterpret_cast<uint2*>(dst + 8 * ca) = e4m3_chunk(a[m], inv);
    *reinterpret_cast<uint2*>(dst + 8 * cb) = e4m3_chunk(b[m], inv);
  }
  __syncthreads();  // every thread has read the old scale
  if (threadIdx.x == 0) *scale_at = s;
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
      !aligned(c->runs, 16) || !aligned(c->free_next, 4) || !aligned(c->status, 4))
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
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
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
  context_plan_kernel<<<kPlanCtas, kPlanThreads, 0, static_cast<cudaStream_t>(stream)>>>(*ctx, add, release, commit);
  return cuda_ok(cudaGetLastError(), "context plan launch") ? DG_OK : DG_ERR_CUDA;
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
  if (s[1] != 0 && !cuda_ok(cudaMemsetAsync(ctx->status + 1, 0, sizeof(int32_t), cs), "context latch clear"))
    return DG_ERR_CUDA;
  if (s[0] != 0) {
    set_last_error_message(s[0] == 1   ? "the context's pool has too few free pages for the batch"
                           : s[0] == 2 ? "the batch has more rows than the context"
                                       : "a length is negative or beyond the context's table");
    return DG_ERR_CAPACITY;
  }
  if (s[1] != 0) {
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
  auto launch = [&](auto kernel, int tokens) {
    kernel<<<(rows + tokens - 1) / tokens, kRopeThreads, 0, cs>>>(
        static_cast<const uint8_t*>(x->data), static_cast<uint8_t*>(out->data), x->row_stride, x->head_stride,
        out->row_stride, out->head_stride, rows, heads, dim, positions, rope->freq, rope->rot, rope->interleaved,
        rope->magnitude);
  };
  // few rows: a CTA per row, for the latency; else four, for the turns
  if (rows <= 4 * sms)
    launch(rope_kernel<1>, 1);
  else
    launch(rope_kernel<4>, 4);
  return cuda_ok(cudaGetLastError(), "rope launch") ? DG_OK : DG_ERR_CUDA;
}

dg_status dg_context_append(const dg_context* ctx, const dg_context_cache* cache, const dg_heads* k,
                            const dg_heads* v, const dg_rope_args* rope, void* stream) {
  dg_status st;
  if ((st = check_context(ctx)) != DG_OK || (st = check_cache(cache, ctx)) != DG_OK) return st;
  if ((st = check_heads(k, cache->heads, cache->dim)) != DG_OK) return st;
  if ((st = check_heads(v, cache->heads, cache->dim)) != DG_OK) return st;
  if (rope != nullptr && (st = check_rope(rope, cache->dim)) != DG_OK) return st;
  if (device_sms() <= 0) return DG_ERR_NO_DEVICE;
  const dim3 grid(DG_CONTEXT_RUNS(ctx->rows, ctx->B), cache->heads, 2);
  const dg_rope_args none = {};
  auto kernel = cache->dim == 128 ? context_append_kernel<128> : context_append_kernel<64>;
  kernel<<<grid, kAppendThreads, 0, static_cast<cudaStream_t>(stream)>>>(*ctx, *cache, *k, *v, rope ? *rope : none,
                                                                         rope != nullptr);
  return cuda_ok(cudaGetLastError(), "context append launch") ? DG_OK : DG_ERR_CUDA;
}

}  // extern "C"
