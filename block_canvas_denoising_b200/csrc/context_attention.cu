// context_attention.cu -- attention of a batch's new rows over the 8-bit
// paged cache: the entry points, and the kernel for few rows per kv head
// (single tokens).
//
// The weight of key n in row i is softmax_n(scale q_i . (s_n k_n)) with E4M3
// codes k_n and the power-of-two scale s_n of the key's page; values
// likewise.  All of it in one pass over the keys with a running maximum and
// sum.  Three things hold in both kernels:
//   - logits are kept in units of log2: x = (q . k) c with c the row's, the
//     page's and the softmax's factors in one float32;
//   - the value scale 2^e of a page goes into the weights, not the values:
//     the running maximum m is over x + e and a weight is 2^(x + e - m + 10),
//     at most 2^10, in float16 (11 significant bits, 2^-34 the smallest), so
//     the values enter the matrix product as codes, which float16 holds
//     exactly; the normaliser sums 2^-e times the float32 weights;
//   - a key that is not seen gets x = -inf and weight 0; values behind a
//     request's last token are zeroed, whatever the page holds there.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "context.h"
#include "context_attention.h"
#include "dg_internal.h"
#include "per_device.h"

namespace dg {

namespace {

constexpr size_t kWsAlign = 256;
constexpr float kWeightLog2 = 10.f;  // weights are at most 2^10

// ---------------------------------------------------------------------------
// few rows: warps on their own, mma.sync over pages
// ---------------------------------------------------------------------------
constexpr int kRowsM = 16;
constexpr int kRowsWarps = 4;
constexpr int kRowsThreads = kRowsWarps * 32;

template <int kDim>
struct RowsCfg {
  static constexpr int kPageBytes = DG_PAGE * kDim;             // codes of one (page, head), k or v
  static constexpr int kStages = kDim == 128 ? 3 : 6;           // pages in flight per warp
  static constexpr int kRing = kRowsWarps * kStages * 2 * kPageBytes;
  static constexpr int kSmem = kRing + 1024 + 1024;
  static constexpr int kPartFloats = kRowsM * (kDim + 2);
};

DG_DEV void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four E4M3 codes to float16 pairs (exact).
DG_DEV void codes_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
DG_DEV uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
DG_DEV uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
DG_DEV uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The power of two f (as its exponent) that brings a row's largest magnitude
// to [2^14, 2^15): bf16 values times f are exact in float16 down to 2^-28 of
// the largest, far below float32 sums of the products.  Returns false for a
// row that holds a value that is not finite.
DG_DEV bool row_exponent(float top, int& e) {
  const int b = static_cast<int>(__float_as_uint(top) >> 23);
  e = b == 0 ? 0 : min(14 - (b - 127), 120);
  return b < 255;
}
// One warp walks its own pages with its own copies in flight and its own
// softmax; the block's four warps meet once per item.  A page (64 keys) is 8
// key tiles of mma.m16n8k16.  Which element of a head is "k index 2t" of an
// instruction is free as long as both operands agree, and so is which key is
// "k index" of the second product: thread t of a quad takes 32 consecutive
// elements (16 at dim 64) of a key, so its operands are whole 16-byte reads
// of the codes as the cache holds them, and the second product takes the
// keys where the first left its results.  Nothing is transposed.
template <int kDim>
__global__ void __launch_bounds__(kRowsThreads, 1)
attention_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ AttnParams p) {
  using Cfg = RowsCfg<kDim>;
  using S = Split<kRowsM, DG_PAGE>;
  constexpr int kSteps = kDim / 16;      // k steps of q . k
  constexpr int kNt = kDim / 8;          // 8-wide output tiles
  constexpr int kSlice = kDim / 4;       // elements of a key held by one thread of a quad
  extern __shared__ uint8_t smem_raw[];
  __shared__ int64_t s_before[DG_MAX_B + 1];
  __shared__ uint64_t s_bars[kRowsWarps][Cfg::kStages][2];
  __shared__ float s_scale[kRowsWarps][Cfg::kStages][2];
  __shared__ float s_m[kRowsWarps][kRowsM], s_l[kRowsWarps][kRowsM];
  __shared__ uint32_t s_last;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* s_o = reinterpret_cast<float*>(ring);  // [warps][16][dim], between items
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;

  if (lane == 0) {
    for (int s = 0; s < Cfg::kStages; ++s) {
      mbar_init(smem_u32(&s_bars[warp][s][0]), 1);
      mbar_init(smem_u32(&s_bars[warp][s][1]), 1);
    }
    fence_mbarrier_init();
  }
  S::totals(p, s_before);
  const int64_t total = s_before[p.B];
  const int64_t even = (total + gridDim.x - 1) / gridDim.x;
  const int64_t per = even > p.min_tiles ? even : p.min_tiles;
  int64_t pos = blockIdx.x * per;
  const int64_t end = min(pos + per, total);
  const uint64_t policy = policy_evict_first();
  int stage = 0;
  uint32_t phase = 0;
  bool ok = true;

  while (pos < end) {
    S it;
    it.find(p, s_before, pos);
    const int64_t item_end = it.begin + it.tiles;
    const int seg = static_cast<int>(min(item_end, end) - pos);
    const int page0 = it.first + static_cast<int>(pos - it.begin);
    const Request& rq = it.q;
    const int mine = seg > warp ? (seg - warp + kRowsWarps - 1) / kRowsWarps : 0;

    // copies: lane l of the warp knows the id and scales of its pages 32 j + l
    int id = 0;
    float ks = 1.f, vs = 1.f;
    auto issue = [&](int n) {
      if ((n & 31) == 0) {
        const int m = n + lane;
        const int pg = page0 + warp + m * kRowsWarps;
        id = -1;
        if (m < mine && pg < p.max_pages) id = p.table[static_cast<size_t>(it.r) * p.max_pages + pg];
        ks = vs = 1.f;
        if (id < 0 || id >= p.pages) {
          id = p.pages;  // outside the tensor: the copy fills zeros
          ks = -1.f;     // and its keys are not seen
        } else {
          ks = p.k_scale[static_cast<size_t>(id) * p.kv_heads + it.h];
          vs = p.v_scale[static_cast<size_t>(id) * p.kv_heads + it.h];
        }
      }
      const int n_id = __shfl_sync(0xffffffffu, id, n & 31);
      const float n_ks = __shfl_sync(0xffffffffu, ks, n & 31), n_vs = __shfl_sync(0xffffffffu, vs, n & 31);
      int st = stage + (n < Cfg::kStages ? n : 0);  // ahead of the reader only before the loop
      if (st >= Cfg::kStages) st -= Cfg::kStages;
      if (lane == 0) {
        s_scale[warp][st][0] = n_ks;
        s_scale[warp][st][1] = n_vs;
        const int y = (n_id * p.kv_heads + it.h) * DG_PAGE;
        const uint32_t dst = smem_u32(ring) + ((warp * Cfg::kStages + st) * 2) * Cfg::kPageBytes;
        const uint32_t kb = smem_u32(&s_bars[warp][st][0]), vb = smem_u32(&s_bars[warp][st][1]);
        mbar_arrive_expect_tx(kb, Cfg::kPageBytes);
        tma_load_2d(dst, &tmK, kb, 0, y, policy);
        mbar_arrive_expect_tx(vb, Cfg::kPageBytes);
        tma_load_2d(dst + Cfg::kPageBytes, &tmV, vb, 0, y, policy);
      }
    };
    for (int n = 0; n < Cfg::kStages && n < mine; ++n) issue(n);

    // this thread's rows g and g + 8 of the item: operands and factor
    uint32_t qf[kSteps][4];
    float fac[2];
    int lo[2], hi[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int64_t rho = static_cast<int64_t>(it.mt) * kRowsM + g + 8 * half;
      const int i = static_cast<int>(rho / p.group), head = it.h * p.group + static_cast<int>(rho % p.group);
      const bool live = i < rq.nq;
      lo[half] = live ? key_lo(p, rq, i) : 1;
      hi[half] = live ? key_hi(rq, i) : 0;
      float x[kSlice];
      float top = 0.f;
      bool finite = true;
#pragma unroll
      for (int c = 0; c < kSlice / 8; ++c) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (live)
          w = *reinterpret_cast<const uint4*>(p.q + (rq.row0 + i) * p.q_row + head * p.q_head + 2 * kSlice * t + 16 * c);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[8 * c + 2 * j] = __uint_as_float(u[j] << 16);
          x[8 * c + 2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float a = fabsf(x[8 * c + j]);
          finite = finite && a <= FLT_MAX;
          top = fmaxf(top, a);
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      int fin = finite;
      fin &= __shfl_xor_sync(0xffffffffu, fin, 1);
      fin &= __shfl_xor_sync(0xffffffffu, fin, 2);
      int e;
      row_exponent(top, e);
      const float f = fin ? pow2i(e) : 0.f;
      fac[half] = fin ? p.scale_log2 * pow2i(-e) : __int_as_float(0x7fc00000);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        qf[s][half] = half2_of(x[4 * s] * f, x[4 * s + 1] * f);
        qf[s][2 + half] = half2_of(x[4 * s + 2] * f, x[4 * s + 3] * f);
      }
    }

    float m[2] = {-FLT_MAX, -FLT_MAX}, l[2] = {0.f, 0.f};
    float o[kNt][4];
#pragma unroll
    for (int j = 0; j < kNt; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

    for (int n = 0; n < mine; ++n) {
      __syncwarp();
      const float ks_n = s_scale[warp][stage][0], vs_n = s_scale[warp][stage][1];
      const uint32_t kbase = smem_u32(ring) + ((warp * Cfg::kStages + stage) * 2) * Cfg::kPageBytes;
      const uint32_t vbase = kbase + Cfg::kPageBytes;
      const int key0 = (page0 + warp + n * kRowsWarps) * DG_PAGE;
      if (ok && !mbar_wait_bounded(smem_u32(&s_bars[warp][stage][0]), phase, p.wait_ns)) ok = false;
      float s[8][4];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
        uint32_t w[kSlice / 4];
        const int row = 8 * j + g;
        if (kDim == 128) {  // chunks 2t, 2t + 1 of a 128-byte row, swizzled by the row
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint4 v = lds128(kbase + row * 128 + (((2 * t + c) ^ (row & 7)) << 4));
            w[4 * c] = v.x; w[4 * c + 1] = v.y; w[4 * c + 2] = v.z; w[4 * c + 3] = v.w;
          }
        } else {  // chunk t of a 64-byte row, swizzled by the row pair
          const uint4 v = lds128(kbase + row * 64 + ((t ^ ((row >> 1) & 3)) << 4));
          w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t b0, b1;
          codes_to_half(w[k], b0, b1);
          mma_16816(s[j], qf[k], b0, b1);
        }
      }
      // logits, weights
      const bool seen = ks_n > 0.f;
      const float e = seen ? static_cast<float>(static_cast<int>(__float_as_uint(vs_n) >> 23) - 127) : 0.f;
      const float inv_vs = seen ? 1.0f / vs_n : 1.f;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float c = fac[half] * ks_n;
        float top = -INFINITY;
        const bool all = seen && lo[half] <= key0 && hi[half] >= key0 + DG_PAGE - 1;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x = s[j][2 * half + k] * c;
            const int key = key0 + 8 * j + 2 * t + k;
            if (!all && (!seen || key < lo[half] || key > hi[half])) x = -INFINITY;
            s[j][2 * half + k] = x;
            top = fmaxf(top, x);
          }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float mn = fmaxf(m[half], top + e);
        const float shrink = exp2f(m[half] - mn);
        m[half] = mn;
        const float off = e - mn + kWeightLog2;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float w = exp2_fast(s[j][2 * half + k] + off);
            s[j][2 * half + k] = w;
            sum += w;
          }
        }
        l[half] = l[half] * shrink + sum * inv_vs;
#pragma unroll
        for (int j = 0; j < kNt; ++j) {
          o[j][2 * half] *= shrink;
          o[j][2 * half + 1] *= shrink;
        }
      }
      if (ok && !mbar_wait_bounded(smem_u32(&s_bars[warp][stage][1]), phase, p.wait_ns)) ok = false;
      const int there = rq.len - key0;  // tokens of this page that exist
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t a[4];
        a[0] = half2_of(s[2 * i][0], s[2 * i][1]);
        a[1] = half2_of(s[2 * i][2], s[2 * i][3]);
        a[2] = half2_of(s[2 * i + 1][0], s[2 * i + 1][1]);
        a[3] = half2_of(s[2 * i + 1][2], s[2 * i + 1][3]);
        uint32_t w[4][kDim / 32];  // keys 2t, 2t + 1, 2t + 8, 2t + 9 of 16: dim / 8 elements each
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = 16 * i + 2 * t + (k & 1) + 8 * (k >> 1);
          if (kDim == 128) {
            const uint4 v = lds128(vbase + row * 128 + ((g ^ (row & 7)) << 4));
            w[k][0] = v.x; w[k][1] = v.y; w[k][kDim / 32 - 2] = v.z; w[k][kDim / 32 - 1] = v.w;
          } else {
            const uint2 v = lds64(vbase + row * 64 + ((((g >> 1) ^ ((row >> 1) & 3)) << 4) | ((g & 1) << 3)));
            w[k][0] = v.x; w[k][1] = v.y;
          }
          if (row >= there) {
#pragma unroll
            for (int j = 0; j < kDim / 32; ++j) w[k][j] = 0;
          }
        }
#pragma unroll
        for (int j = 0; j < kDim / 32; ++j) {
          // bytes (key 2t, key 2t + 1) of each of 4 elements
          uint32_t b[4][2];
          codes_to_half(__byte_perm(w[0][j], w[1][j], 0x5140), b[0][0], b[1][0]);
          codes_to_half(__byte_perm(w[0][j], w[1][j], 0x7362), b[2][0], b[3][0]);
          codes_to_half(__byte_perm(w[2][j], w[3][j], 0x5140), b[0][1], b[1][1]);
          codes_to_half(__byte_perm(w[2][j], w[3][j], 0x7362), b[2][1], b[3][1]);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_16816(o[4 * j + k], a, b[k][0], b[k][1]);
        }
      }
      __syncwarp();
      if (n + Cfg::kStages < mine) issue(n + Cfg::kStages);
      if (++stage == Cfg::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }

    // the warps meet: (m, l, o) of each through shared memory (the ring is
    // idle: every copy issued for this item has been waited for)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
      l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
    }
    __syncthreads();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int row = g + 8 * half;
      float* dst = s_o + (warp * kRowsM + row) * kDim + kSlice * t;
#pragma unroll
      for (int j = 0; j < kNt; ++j) {  // columns 2t, 2t + 1 of tile j are elements slice + j, slice + dim / 8 + j
        dst[j] = o[j][2 * half];
        dst[kNt + j] = o[j][2 * half + 1];
      }
      if (t == 0) {
        s_m[warp][row] = m[half];
        s_l[warp][row] = l[half];
      }
    }
    __syncthreads();

    const bool whole = it.begin >= blockIdx.x * per && item_end <= end;
    const int c0 = static_cast<int>(it.begin / per), parts = static_cast<int>((item_end - 1) / per) - c0 + 1;
    float* part = p.part + static_cast<size_t>(2 * blockIdx.x + (static_cast<int>(blockIdx.x) == c0 ? 1 : 0)) * Cfg::kPartFloats;
    constexpr int kChunks = kRowsM * kDim / 8;
    auto store = [&](int row, int d0, const float (&x)[8], float top, float sum) {
      const int64_t rho = static_cast<int64_t>(it.mt) * kRowsM + row;
      const int i = static_cast<int>(rho / p.group), head = it.h * p.group + static_cast<int>(rho % p.group);
      if (i >= rq.nq) return;
      const float inv = sum == 0.f ? 0.f : 1.0f / sum;
      uint32_t u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * j] * inv, x[2 * j + 1] * inv);
        u[j] = *reinterpret_cast<const uint32_t*>(&b);
      }
      *reinterpret_cast<uint4*>(p.out + (rq.row0 + i) * p.out_row + head * p.out_head + 2 * d0) =
          make_uint4(u[0], u[1], u[2], u[3]);
      if (p.lse != nullptr && d0 == 0)
        p.lse[static_cast<size_t>(rq.row0 + i) * (p.kv_heads * p.group) + head] =
            sum == 0.f ? -INFINITY : (top - kWeightLog2 + log2f(sum)) * kLn2;
    };
    for (int c = threadIdx.x; c < kChunks; c += kRowsThreads) {
      const int row = c / (kDim / 8), d0 = (c % (kDim / 8)) * 8;
      float top = s_m[0][row];
#pragma unroll
      for (int w = 1; w < kRowsWarps; ++w) top = fmaxf(top, s_m[w][row]);
      float sum = 0.f, x[8] = {};
#pragma unroll
      for (int w = 0; w < kRowsWarps; ++w) {
        const float f = join_weight(s_m[w][row], top);
        sum += s_l[w][row] * f;
        const float4 a = *reinterpret_cast<const float4*>(s_o + (w * kRowsM + row) * kDim + d0);
        const float4 b = *reinterpret_cast<const float4*>(s_o + (w * kRowsM + row) * kDim + d0 + 4);
        x[0] += a.x * f; x[1] += a.y * f; x[2] += a.z * f; x[3] += a.w * f;
        x[4] += b.x * f; x[5] += b.y * f; x[6] += b.z * f; x[7] += b.w * f;
      }
      if (whole) {
        store(row, d0, x, top, sum);
      } else {
        float4* dst = reinterpret_cast<float4*>(part + row * kDim + d0);
        dst[0] = make_float4(x[0], x[1], x[2], x[3]);
        dst[1] = make_float4(x[4], x[5], x[6], x[7]);
        if (d0 == 0) {
          part[kRowsM * kDim + row] = top;
          part[kRowsM * kDim + kRowsM + row] = sum;
        }
      }
    }
    if (!whole) {
      // the CTA that finishes an item's last part joins them, in split order
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        const uint32_t before = atomicAdd(p.tickets + c0, 1u);
        s_last = before + 1 == static_cast<uint32_t>(parts);
        if (s_last) p.tickets[c0] = 0;
        __threadfence();
      }
      __syncthreads();
      if (s_last) {
        auto part_of = [&](int i) {
          return p.part + static_cast<size_t>(2 * (c0 + i) + (i == 0 ? 1 : 0)) * Cfg::kPartFloats;
        };
        for (int c = threadIdx.x; c < kChunks; c += kRowsThreads) {
          const int row = c / (kDim / 8), d0 = (c % (kDim / 8)) * 8;
          float top = -FLT_MAX;
          for (int i = 0; i < parts; ++i) top = fmaxf(top, __ldcg(part_of(i) + kRowsM * kDim + row));
          float sum = 0.f, x[8] = {};
          for (int i = 0; i < parts; ++i) {
            const float* src = part_of(i);
            const float f = join_weight(__ldcg(src + kRowsM * kDim + row), top);
            sum += __ldcg(src + kRowsM * kDim + kRowsM + row) * f;
            const float4 a = __ldcg(reinterpret_cast<const float4*>(src + row * kDim + d0));
            const float4 b = __ldcg(reinterpret_cast<const float4*>(src + row * kDim + d0 + 4));
            x[0] += a.x * f; x[1] += a.y * f; x[2] += a.z * f; x[3] += a.w * f;
            x[4] += b.x * f; x[5] += b.y * f; x[6] += b.z * f; x[7] += b.w * f;
          }
          store(row, d0, x, top, sum);
        }
      }
    }
    fence_proxy_async();  // the ring goes back to the copies
    __syncthreads();
    pos += seg;
  }
  if (!ok && lane == 0) atomicOr(p.err, kErrWaitContext);
}

template <int kDim>
int rows_grid() {
  static PerDevice<int> cache;
  int dev = -1, n = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  const bool got = cache.get(dev, [](int* v) {
    if (cudaFuncSetAttribute(attention_rows_kernel<kDim>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             RowsCfg<kDim>::kSmem) != cudaSuccess)
      return false;
    int per_sm = 0, sms = device_sms();
    if (sms <= 0 || cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, attention_rows_kernel<kDim>, kRowsThreads,
                                                                  RowsCfg<kDim>::kSmem) != cudaSuccess || per_sm < 1)
      return false;
    *v = per_sm * sms;
    return true;
  }, &n);
  return got ? n : -1;
}

// Workspace: the fault latch, the tickets, the split items, the parts.  Sized for both
// kernels, so that one workspace serves every batch of a shape.
struct AttnWs {
  int rows_grid, tiles_grid;
  size_t tickets, splits, part, total;
};
bool attn_ws(int dim, AttnWs* w) {
  w->rows_grid = dim == 128 ? rows_grid<128>() : rows_grid<64>();
  w->tiles_grid = tiles_grid(dim);
  if (w->rows_grid < 1 || w->tiles_grid < 1) return false;
  const size_t rows_floats = dim == 128 ? RowsCfg<128>::kPartFloats : RowsCfg<64>::kPartFloats;
  const size_t a = static_cast<size_t>(w->rows_grid) * rows_floats, b = w->tiles_grid * tiles_part_floats(dim);
  const int grid = w->rows_grid > w->tiles_grid ? w->rows_grid : w->tiles_grid;
  w->tickets = kWsAlign;
  auto up = [](size_t n) { return (n + kWsAlign - 1) / kWsAlign * kWsAlign; };
  w->splits = w->tickets + up(static_cast<size_t>(grid) * 4);
  w->part = w->splits + up(static_cast<size_t>(grid) * tiles_split_bytes());
  w->total = w->part + 2 * sizeof(float) * (a > b ? a : b);
  return true;
}

bool shape_ok(int64_t rows, int64_t q_heads, int64_t kv_heads, int dim) {
  return rows >= 1 && rows <= kContextMaxRows && kv_heads >= 1 && kv_heads <= 1024 && q_heads >= kv_heads &&
         q_heads % kv_heads == 0 && q_heads / kv_heads <= 1024 && (dim == 64 || dim == 128) &&
         rows * (q_heads / kv_heads) <= 0x7fffffffll;
}

}  // namespace

}  // namespace dg

using namespace dg;

extern "C" {

size_t dg_context_workspace_size(int32_t rows, int32_t q_heads, int32_t kv_heads, int32_t dim) {
  if (!shape_ok(rows, q_heads, kv_heads, dim)) return 0;
  if (device_sms() <= 0) return 0;
  AttnWs ws;
  return attn_ws(dim, &ws) ? ws.total : 0;
}

dg_status dg_context_attention(const dg_context* ctx, const dg_context_cache* cache, const dg_heads* q,
                               const dg_heads* out, int32_t q_heads, float scale, const uint8_t* causal,
                               int32_t window, int32_t max_new, float* lse, void* workspace, size_t ws_bytes,
                               void* stream) {
  dg_status st;
  if ((st = check_context(ctx)) != DG_OK || (st = check_cache(cache, ctx)) != DG_OK) return st;
  if (!shape_ok(ctx->rows, q_heads, cache->heads, cache->dim)) return DG_ERR_UNSUPPORTED_SHAPE;
  if ((st = check_heads(q, q_heads, cache->dim)) != DG_OK || (st = check_heads(out, q_heads, cache->dim)) != DG_OK)
    return st;
  if (q->data == out->data || !(scale >= 0.f && scale <= FLT_MAX) || window < 0 || max_new < 0 ||
      (reinterpret_cast<uintptr_t>(lse) & 3) != 0)
    return DG_ERR_INVALID_ARG;
  if (device_sms() <= 0) return DG_ERR_NO_DEVICE;
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & (kWsAlign - 1)) != 0) return DG_ERR_INVALID_ARG;
  const int dim = cache->dim;
  AttnWs ws;
  if (!attn_ws(dim, &ws)) {
    set_last_error_message("no CTA of a context attention kernel fits on this device");
    return DG_ERR_CUDA;
  }
  if (ws_bytes < ws.total) return DG_ERR_WORKSPACE;

  AttnParams p;
  memset(&p, 0, sizeof(p));
  p.table = ctx->table;
  p.lens = ctx->lens;
  p.start = ctx->start;
  p.B = ctx->B;
  p.max_pages = ctx->max_pages;
  p.pages = ctx->pages;
  p.rows = ctx->rows;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.kv_heads = cache->heads;
  p.group = q_heads / cache->heads;
  p.q = static_cast<const uint8_t*>(q->data);
  p.out = static_cast<uint8_t*>(out->data);
  p.q_row = 2 * q->row_stride;
  p.q_head = 2 * q->head_stride;
  p.out_row = 2 * out->row_stride;
  p.out_head = 2 * out->head_stride;
  p.lse = lse;
  p.scale_log2 = static_cast<float>((scale == 0.f ? 1.0 / sqrt(static_cast<double>(dim)) : static_cast<double>(scale)) *
                                    1.4426950408889634);
  p.causal = causal;
  p.window = window;
  uint8_t* wsb = static_cast<uint8_t*>(workspace);
  p.err = reinterpret_cast<uint32_t*>(wsb);
  p.tickets = reinterpret_cast<uint32_t*>(wsb + ws.tickets);
  p.splits = wsb + ws.splits;
  p.part = reinterpret_cast<float*>(wsb + ws.part);
  p.wait_ns = kDefaultWaitNs;

  CUtensorMap tmK, tmV;
  const uint64_t crows = static_cast<uint64_t>(cache->pages) * cache->heads * DG_PAGE;
  const auto sw = dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if (!encode_2d(&tmK, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, sw, cache->k, dim, crows, dim, DG_PAGE) ||
      !encode_2d(&tmV, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, sw, cache->v, dim, crows, dim, DG_PAGE)) {
    set_last_error_message("context attention: tensor map of the cache");
    return DG_ERR_CUDA;
  }
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  // One row tile of the rows kernel is 16 rows; the tiles kernel works on 256
  // whether they are there or not.
  const int64_t most = static_cast<int64_t>(max_new > 0 && max_new < ctx->rows ? max_new : ctx->rows) * p.group;
  if (most > kRowsM) {
    p.min_tiles = 1;
    return cuda_ok(launch_attention_tiles(dim, tmK, tmV, p, ws.tiles_grid, cs), "context attention launch") ? DG_OK
                                                                                                       : DG_ERR_CUDA;
  }
  p.min_tiles = kRowsWarps;
  if (dim == 128)
    attention_rows_kernel<128><<<ws.rows_grid, kRowsThreads, RowsCfg<128>::kSmem, cs>>>(tmK, tmV, p);
  else
    attention_rows_kernel<64><<<ws.rows_grid, kRowsThreads, RowsCfg<64>::kSmem, cs>>>(tmK, tmV, p);
  return cuda_ok(cudaGetLastError(), "context attention launch") ? DG_OK : DG_ERR_CUDA;
}

}  // extern "C"
