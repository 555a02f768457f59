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
// kNt: the rows of an item, in eights.
template <int kDim, int kNt>
struct RowsCfg {
  static constexpr int kM = 8 * kNt;
  // Warps of a block.  What bounds it is registers (97 to 160 a thread) and
  // the warps' pages in shared memory.
  static constexpr int kWarps = kNt == 1 ? (kDim == 128 ? 12 : 16) : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kPageBytes = DG_PAGE * kDim;             // codes of one (page, head), k or v
  // A page of keys and one of values per warp.  The next keys are asked for
  // as soon as these are multiplied, the next values likewise, so one of the
  // two is always on its way: 64 KB or more in flight on an SM.
  static constexpr int kRing = kWarps * 2 * kPageBytes;
  static constexpr int kSmem = kRing + 1024;
  static constexpr int kPartFloats = kM * (kDim + 2);
  static_assert(kRing >= kWarps * kM * kDim * 4 && kSmem <= 220 * 1024, "the warps meet in the ring");
};

// Not volatile, like the conversions: the compiler is free to put independent
// products between dependent ones.
DG_DEV void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
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
DG_DEV uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The transpose of an 8 x 8 matrix of 16-bit elements, two per thread.
DG_DEV uint32_t transpose8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

// One warp walks its own pages with its own copies in flight and its own
// softmax; the block's warps meet once per item.  A page (64 keys) is four key
// tiles of mma.m16n8k16 with the keys as the 16 rows and the item's rows as
// the 8 columns: S^T = K Q^T and O^T = V^T P^T, so that no more than 8 of
// those are paid for where there are 4 (with the rows as the 16: twice the
// products and accumulators, 8 warps on an SM, and 2.4 TB/s of cache).
// Which element of a head is "k index 2t" of an instruction is free as long
// as both operands agree, and so is which element is which row of O^T: thread
// t of a quad takes dim / 4 consecutive elements of a key, and quad g dim / 8
// of a value, so operands are whole 16-byte reads of the codes as the cache
// holds them.  Between the products P is transposed 8 x 8 at a time.
// Measured (128-wide heads): one token of 32 requests over 1000 to 9000 tokens
// (8 kv heads, 4 query heads each) in 61.9 us, 5.5 TB/s of cache, 0.84 of a plain
// copy's rate: bound by HBM.  One token over 4096 (4 kv heads) in 13 us: a
// chain of some ten dependent reads (lengths, table, scales, page, the other
// CTAs' parts) of 0.5 to 1 us each.
template <int kDim, int kNt>
__global__ void __launch_bounds__(RowsCfg<kDim, kNt>::kThreads, 1)
attention_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ AttnParams p) {
  using Cfg = RowsCfg<kDim, kNt>;
  using S = Split<Cfg::kM, DG_PAGE, 2 * Cfg::kWarps>;  // an item costs about two pages a warp
  constexpr int kM = Cfg::kM, kWarps = Cfg::kWarps;
  constexpr int kSteps = kDim / 16;      // k steps of q . k
  constexpr int kSlice = kDim / 4;       // elements of a key held by one thread of a quad
  constexpr int kDt = kDim / 16;         // 16-row tiles of O^T
  constexpr int kVw = kDim / 32;         // words of a value held by a thread
  extern __shared__ uint8_t smem_raw[];
  __shared__ int64_t s_before[DG_MAX_B + 1];
  __shared__ uint64_t s_bars[kWarps][2];
  __shared__ float s_m[kWarps][kM], s_l[kWarps][kM];
  __shared__ uint32_t s_last;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* s_o = reinterpret_cast<float*>(ring);  // [warps][kM][dim], between items
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;

  if (lane == 0) {
    mbar_init(smem_u32(&s_bars[warp][0]), 1);
    mbar_init(smem_u32(&s_bars[warp][1]), 1);
    fence_mbarrier_init();
  }
  wait_for_previous_kernel();
  allow_next_kernel();
  S::totals(p, s_before);
  const int64_t total = s_before[p.B];
  const int64_t even = quotient(total + gridDim.x - 1, gridDim.x);
  const int64_t per = even > p.min_tiles ? even : p.min_tiles;
  int64_t pos = blockIdx.x * per;
  const int64_t end = min(pos + per, total);
  const uint64_t policy = policy_evict_first();
  uint8_t* k_page = ring + warp * 2 * Cfg::kPageBytes;
  uint8_t* v_page = k_page + Cfg::kPageBytes;
  const uint32_t k_bar = smem_u32(&s_bars[warp][0]), v_bar = smem_u32(&s_bars[warp][1]);
  uint32_t phase = 0;
  bool ok = true;

  while (pos < end) {
    S it;
    it.find(p, s_before, pos);
    pos = max(pos, it.begin);  // the units before an item's first tile stand for its fixed cost
    if (pos >= end) break;
    const int64_t item_end = it.begin + it.tiles;
    const int seg = static_cast<int>(min(item_end, end) - pos);
    const int page0 = it.first + static_cast<int>(pos - it.begin);
    const Request& rq = it.q;
    const int mine = seg > warp ? (seg - warp + kWarps - 1) / kWarps : 0;

    // ids and scales of the warp's pages n0 .. n0 + 31, one per lane
    int id = 0;
    float ks = 1.f, vs = 1.f;
    auto look_up = [&](int n0) {
      const int n = n0 + lane, pg = page0 + warp + n * kWarps;
      id = -1;
      if (n < mine && pg < p.max_pages) id = p.table[static_cast<size_t>(it.r) * p.max_pages + pg];
      if (id < 0 || id >= p.pages) {
        id = p.pages;  // outside the tensor: the copy fills zeros
        ks = -1.f;     // and its keys are not seen
        vs = 1.f;
      } else {
        ks = p.k_scale[static_cast<size_t>(id) * p.kv_heads + it.h];
        vs = p.v_scale[static_cast<size_t>(id) * p.kv_heads + it.h];
      }
    };
    // all lanes; only page n of the looked up ones
    auto copy = [&](const CUtensorMap* map, uint8_t* to, uint32_t bar, int n) {
      const int y = (__shfl_sync(0xffffffffu, id, n & 31) * p.kv_heads + it.h) * DG_PAGE;
      if (lane == 0 && ok) {
        mbar_arrive_expect_tx(bar, Cfg::kPageBytes);
        tma_load_2d(smem_u32(to), map, bar, 0, y, policy);
      }
    };
    if (mine > 0) {
      look_up(0);
      copy(&tmK, k_page, k_bar, 0);
      copy(&tmV, v_page, v_bar, 0);
    }

    // queries: thread (g, t) holds its slice of rows g (and g + 8) as operands;
    // thread t is in charge of the softmax of rows 2t, 2t + 1 (and 8 further)
    uint32_t qf[kNt][kSteps][2];
    float fac[kNt][2];
    int lo[kNt][2], hi[kNt][2];
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) {
      const uint32_t rho = static_cast<uint32_t>(it.mt) * kM + 8 * nt + g;
      const int i = static_cast<int>(rho / static_cast<uint32_t>(p.group));
      const int head = it.h * p.group + static_cast<int>(rho - static_cast<uint32_t>(i) * p.group);
      const bool live = i < rq.nq;
      float x[kSlice];
      float top = 0.f;
      int fin = 1;
#pragma unroll
      for (int c = 0; c < kSlice / 8; ++c) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (live)
          w = *reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(rq.row0 + i) * p.q_row + head * p.q_head +
                                              2 * kSlice * t + 16 * c);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[8 * c + 2 * j] = __uint_as_float(u[j] << 16);
          x[8 * c + 2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float a = fabsf(x[8 * c + j]);
          fin &= a <= FLT_MAX;
          top = fmaxf(top, a);
        }
      }
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        fin &= __shfl_xor_sync(0xffffffffu, fin, d);
      }
      // The power of two that brings the row's largest magnitude to [2^14,
      // 2^15): bf16 values times it are exact in float16 down to 2^-28 of the
      // largest, far below the float32 sums of the products.
      const int b = static_cast<int>(__float_as_uint(top) >> 23);
      const int e = b == 0 ? 0 : min(14 - (b - 127), 120);
      const float f = fin ? pow2i(e) : 0.f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        qf[nt][s][0] = half2_of(x[4 * s] * f, x[4 * s + 1] * f);
        qf[nt][s][1] = half2_of(x[4 * s + 2] * f, x[4 * s + 3] * f);
      }
      // a row that holds a value that is not finite: NaN for all its logits
      const float mine_fac = fin ? p.scale_log2 * pow2i(-e) : __int_as_float(0x7fc00000);
      const int my_lo = live ? key_lo(p, rq, i) : 0, my_hi = live ? key_hi(rq, i) : 0x7FFFFFF0;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        fac[nt][k] = __shfl_sync(0xffffffffu, mine_fac, 4 * (2 * t + k));
        lo[nt][k] = __shfl_sync(0xffffffffu, my_lo, 4 * (2 * t + k));
        hi[nt][k] = __shfl_sync(0xffffffffu, my_hi, 4 * (2 * t + k));
      }
    }

    float m[kNt][2], l[kNt][2], o[kNt][kDt][4];
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) {
      m[nt][0] = m[nt][1] = -FLT_MAX;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int d = 0; d < kDt; ++d) o[nt][d][0] = o[nt][d][1] = o[nt][d][2] = o[nt][d][3] = 0.f;
    }

    for (int n = 0; n < mine; ++n) {
      const float ks_n = __shfl_sync(0xffffffffu, ks, n & 31), vs_n = __shfl_sync(0xffffffffu, vs, n & 31);
      const int key0 = (page0 + warp + n * kWarps) * DG_PAGE;
      const bool more = n + 1 < mine;
      if (ok && !mbar_wait_bounded(k_bar, phase, p.wait_ns)) ok = false;
      // S^T: s[nt][i] = keys 16 i + g (elements 0, 1: rows 2t, 2t + 1) and 16 i + g + 8 (2, 3)
      float s[kNt][4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt) s[nt][i][0] = s[nt][i][1] = s[nt][i][2] = s[nt][i][3] = 0.f;
        uint32_t w[2][kSlice / 4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int row = 16 * i + 8 * k + g;
#pragma unroll
          for (int c = 0; c < kSlice / 16; ++c) {
            // dim 128: chunks 2t, 2t + 1 of a 128-byte row, swizzled by the row;
            // dim 64: chunk t of a 64-byte row, swizzled by the row pair
            const uint4 v = *reinterpret_cast<const uint4*>(
                k_page + (kDim == 128 ? row * 128 + (((2 * t + c) ^ (row & 7)) << 4) : row * 64 + ((t ^ ((row >> 1) & 3)) << 4)));
            w[k][4 * c] = v.x; w[k][4 * c + 1] = v.y; w[k][4 * c + 2] = v.z; w[k][4 * c + 3] = v.w;
          }
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t a[4];
          codes_to_half(w[0][k], a[0], a[2]);
          codes_to_half(w[1][k], a[1], a[3]);
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt) mma_16816(s[nt][i], a, qf[nt][k][0], qf[nt][k][1]);
        }
      }
      __syncwarp();
      const bool turn = more && ((n + 1) & 31) == 0;  // the next page is of the next 32
      if (more && !turn) copy(&tmK, k_page, k_bar, n + 1);
      // logits, weights
      const bool seen = ks_n > 0.f;
      const float ve = seen ? static_cast<float>(static_cast<int>(__float_as_uint(vs_n) >> 23) - 127) : 0.f;
      bool all = seen;
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) {
#pragma unroll
        for (int k = 0; k < 2; ++k) all = all && lo[nt][k] <= key0 && hi[nt][k] >= key0 + DG_PAGE - 1;
      }
      all = __all_sync(0xffffffffu, all);
      uint32_t pt[kNt][8];  // P^T as the second product's operand: keys 8 j + 2t, + 1 of row g
      bool moved = false;
      float shrink[kNt][2];
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float c = fac[nt][k] * ks_n;
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float x = s[nt][i][2 * h + k] * c;
              if (!all) {
                const int key = key0 + 16 * i + 8 * h + g;
                if (!seen || key < lo[nt][k] || key > hi[nt][k]) x = -INFINITY;
              }
              s[nt][i][2 * h + k] = x;
              top = fmaxf(top, x);
            }
          }
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          const float mn = fmaxf(m[nt][k], top + ve);
          shrink[nt][k] = exp2f(m[nt][k] - mn);
          moved = moved || mn != m[nt][k];
          m[nt][k] = mn;
          const float off = ve - mn + kWeightLog2;
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float w = exp2_fast(s[nt][i][2 * h + k] + off);
              s[nt][i][2 * h + k] = w;
              sum += w;
            }
          }
          l[nt][k] = l[nt][k] * shrink[nt][k] + sum * pow2i(-static_cast<int>(ve));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          pt[nt][2 * i] = transpose8(half2_of(s[nt][i][0], s[nt][i][1]));
          pt[nt][2 * i + 1] = transpose8(half2_of(s[nt][i][2], s[nt][i][3]));
        }
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt) {
#pragma unroll
          for (int d = 0; d < kDt; ++d) {
            o[nt][d][0] *= shrink[nt][0];
            o[nt][d][1] *= shrink[nt][1];
            o[nt][d][2] *= shrink[nt][0];
            o[nt][d][3] *= shrink[nt][1];
          }
        }
      }
      if (ok && !mbar_wait_bounded(v_bar, phase, p.wait_ns)) ok = false;
      const int there = rq.len - key0;  // tokens of this page that exist
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[4][kVw];  // keys 2t, 2t + 1, 2t + 8, 2t + 9 of 16: dim / 8 elements each
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = 16 * i + 2 * t + (k & 1) + 8 * (k >> 1);
          if (kDim == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(v_page + row * 128 + ((g ^ (row & 7)) << 4));
            w[k][0] = v.x; w[k][1] = v.y; w[k][kVw - 2] = v.z; w[k][kVw - 1] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(
                v_page + row * 64 + ((((g >> 1) ^ ((row >> 1) & 3)) << 4) | ((g & 1) << 3)));
            w[k][0] = v.x; w[k][1] = v.y;
          }
        }
        if (there < DG_PAGE) {  // behind the last token: zeros, whatever is there
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (16 * i + 2 * t + (k & 1) + 8 * (k >> 1) >= there) {
#pragma unroll
              for (int j = 0; j < kVw; ++j) w[k][j] = 0;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < kVw; ++j) {
          // rows g and g + 8 of tile d are elements 2d and 2d + 1 of the quad's dim / 8
          uint32_t a[2][4];
          codes_to_half(__byte_perm(w[0][j], w[1][j], 0x5140), a[0][0], a[0][1]);
          codes_to_half(__byte_perm(w[0][j], w[1][j], 0x7362), a[1][0], a[1][1]);
          codes_to_half(__byte_perm(w[2][j], w[3][j], 0x5140), a[0][2], a[0][3]);
          codes_to_half(__byte_perm(w[2][j], w[3][j], 0x7362), a[1][2], a[1][3]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) mma_16816(o[nt][2 * j + k], a[k], pt[nt][2 * i], pt[nt][2 * i + 1]);
          }
        }
      }
      __syncwarp();
      if (turn) {
        look_up(n + 1);
        copy(&tmK, k_page, k_bar, n + 1);
      }
      if (more) copy(&tmV, v_page, v_bar, n + 1);
      if (ok) phase ^= 1u;
    }

    // the warps meet: (m, l, o) of each through shared memory (the ring is
    // idle: every copy issued for this item has been waited for)
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], d);
      }
    }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = 8 * nt + 2 * t + k;
        float* dst = s_o + (warp * kM + row) * kDim + 2 * kDt * g;
#pragma unroll
        for (int d = 0; d < kDt; ++d) *reinterpret_cast<float2*>(dst + 2 * d) = make_float2(o[nt][d][k], o[nt][d][2 + k]);
        if (g == 0) {
          s_m[warp][row] = m[nt][k];
          s_l[warp][row] = l[nt][k];
        }
      }
    }
    __syncthreads();

    const bool whole = pos == it.begin && item_end <= end;
    const int c0 = static_cast<int>(quotient(it.begin, per)), parts = static_cast<int>(quotient(item_end - 1, per)) - c0 + 1;
    float* part = p.part + static_cast<size_t>(2 * blockIdx.x + (static_cast<int>(blockIdx.x) == c0 ? 1 : 0)) * Cfg::kPartFloats;
    constexpr int kChunks = kM * kDim / 8;
    auto store = [&](int row, int d0, const float (&x)[8], float top, float sum) {
      const uint32_t rho = static_cast<uint32_t>(it.mt) * kM + row;
      const int i = static_cast<int>(rho / static_cast<uint32_t>(p.group));
      const int head = it.h * p.group + static_cast<int>(rho - static_cast<uint32_t>(i) * p.group);
      if (i >= rq.nq) return;
      const float inv = sum == 0.f ? 0.f : 1.0f / sum;
      uint32_t u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * j] * inv, x[2 * j + 1] * inv);
        u[j] = *reinterpret_cast<const uint32_t*>(&b);
      }
      *reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(rq.row0 + i) * p.out_row + head * p.out_head + 2 * d0) =
          make_uint4(u[0], u[1], u[2], u[3]);
      if (p.lse != nullptr && d0 == 0)
        p.lse[static_cast<size_t>(rq.row0 + i) * (p.kv_heads * p.group) + head] =
            sum == 0.f ? -INFINITY : (top - kWeightLog2 + log2f(sum)) * kLn2;
    };
    for (int c = threadIdx.x; c < kChunks; c += Cfg::kThreads) {
      const int row = c / (kDim / 8), d0 = (c % (kDim / 8)) * 8;
      float top = s_m[0][row];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w][row]);
      float sum = 0.f, x[8] = {};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = join_weight(s_m[w][row], top);
        sum += s_l[w][row] * f;
        const float4 a = *reinterpret_cast<const float4*>(s_o + (w * kM + row) * kDim + d0);
        const float4 b = *reinterpret_cast<const float4*>(s_o + (w * kM + row) * kDim + d0 + 4);
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
          part[kM * kDim + row] = top;
          part[kM * kDim + kM + row] = sum;
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
        constexpr int kAtOnce = 8;
        for (int c = threadIdx.x; c < kChunks; c += Cfg::kThreads) {
          const int row = c / (kDim / 8), d0 = (c % (kDim / 8)) * 8;
          float top = -FLT_MAX, sum = 0.f, x[8] = {};
          for (int i0 = 0; i0 < parts; i0 += kAtOnce) {  // every read of some parts before the first use
            float mi[kAtOnce], li[kAtOnce];
            float4 ai[kAtOnce], bi[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
              const float* src = part_of(min(i0 + i, parts - 1));
              mi[i] = __ldcg(src + kM * kDim + row);
              li[i] = __ldcg(src + kM * kDim + kM + row);
              ai[i] = __ldcg(reinterpret_cast<const float4*>(src + row * kDim + d0));
              bi[i] = __ldcg(reinterpret_cast<const float4*>(src + row * kDim + d0 + 4));
            }
            float now = top;
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) now = fmaxf(now, mi[i]);
            const float old = join_weight(top, now);
            top = now;
            sum *= old;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= old;
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
              const float f = i0 + i < parts ? join_weight(mi[i], now) : 0.f;  // behind the last part: that one again
              sum += li[i] * f;
              x[0] += ai[i].x * f; x[1] += ai[i].y * f; x[2] += ai[i].z * f; x[3] += ai[i].w * f;
              x[4] += bi[i].x * f; x[5] += bi[i].y * f; x[6] += bi[i].z * f; x[7] += bi[i].w * f;
            }
          }
          store(row, d0, x, top, sum);
        }
      }
    }
    fence_proxy_async();  // the ring goes back to the copies
    __syncthreads();
    pos += seg;
  }
  if (!ok && lane == 0) {
    // It gave up waiting, and has asked for no more pages since.  What it had
    // asked for (keys of this phase, or of the next where these came; values of
    // this one) gets another time to land before the block goes.
    mbar_wait_bounded(k_bar, phase, p.wait_ns);
    mbar_wait_bounded(v_bar, phase, p.wait_ns);
    mbar_wait_bounded(k_bar, phase ^ 1u, p.wait_ns);
  }
  if (!ok) atomicOr(p.err, kErrWaitContext);
}

template <int kDim, int kNt>
int rows_grid() {
  static PerDevice<int> cache;
  int dev = -1, n = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  const bool got = cache.get(dev, [](int* v) {
    using Cfg = RowsCfg<kDim, kNt>;
    if (cudaFuncSetAttribute(attention_rows_kernel<kDim, kNt>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg::kSmem) != cudaSuccess)
      return false;
    int per_sm = 0;
    const int sms = device_sms();
    if (sms <= 0 || cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, attention_rows_kernel<kDim, kNt>,
                                                                  Cfg::kThreads, Cfg::kSmem) != cudaSuccess || per_sm < 1)
      return false;
    *v = per_sm * sms;
    return true;
  }, &n);
  return got ? n : -1;
}

// Workspace: the fault latch, the tickets, the split items, the parts.  Sized
// for all kernels, so that one workspace serves every batch of a shape; the
// tickets' place, which has to stay zero between calls, is the same for every
// shape.
constexpr int kMaxGrid = 1024;
struct AttnWs {
  int grid8, grid16, tiles_grid;  // resident CTAs of the rows kernels and of the tiles kernel
  size_t tickets, splits, part, total;
};
template <int kDim>
bool attn_ws(AttnWs* w) {
  w->grid8 = rows_grid<kDim, 1>();
  w->grid16 = rows_grid<kDim, 2>();
  w->tiles_grid = tiles_grid(kDim);
  if (w->grid8 < 1 || w->grid16 < 1 || w->tiles_grid < 1) return false;
  if (w->grid8 > kMaxGrid || w->grid16 > kMaxGrid || w->tiles_grid > kMaxGrid) return false;
  auto up = [](size_t n) { return (n + kWsAlign - 1) / kWsAlign * kWsAlign; };
  auto most = [](size_t a, size_t b) { return a > b ? a : b; };
  const size_t floats = most(w->grid8 * size_t(RowsCfg<kDim, 1>::kPartFloats),
                             most(w->grid16 * size_t(RowsCfg<kDim, 2>::kPartFloats), w->tiles_grid * tiles_part_floats(kDim)));
  w->tickets = kWsAlign;
  w->splits = w->tickets + up(kMaxGrid * 4);
  w->part = w->splits + up(kMaxGrid * tiles_split_bytes());
  w->total = w->part + 2 * sizeof(float) * floats;
  return true;
}
bool attn_ws(int dim, AttnWs* w) { return dim == 128 ? attn_ws<128>(w) : attn_ws<64>(w); }

template <int kDim>
cudaError_t launch_rows(const CUtensorMap& tmK, const CUtensorMap& tmV, const AttnParams& p, bool eight, const AttnWs& ws,
                        cudaStream_t stream) {
  if (eight)
    return launch_context(attention_rows_kernel<kDim, 1>, dim3(ws.grid8), RowsCfg<kDim, 1>::kThreads,
                          RowsCfg<kDim, 1>::kSmem, stream, tmK, tmV, p);
  return launch_context(attention_rows_kernel<kDim, 2>, dim3(ws.grid16), RowsCfg<kDim, 2>::kThreads,
                        RowsCfg<kDim, 2>::kSmem, stream, tmK, tmV, p);
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
  // Rows a kv head has in one request at most: the rows kernel takes 8 or 16
  // at a time and reads the keys again for each, the tiles kernel takes 256
  // whether they are there or not.  Microseconds of eights / sixteens / tiles:
  //   rows                              8              16             32             48
  //   32 requests x 5000 tokens     60  76 162    106  84 170    206 159 181    296 235 182
  //   256 requests x 300 tokens     92 120 249    175 121 271    343 238 287    518 356 262
  //   1 request x 4096 tokens       12  14  26     12  15  26     13  15  26     14  15  26
  // (8 kv heads x 128; 4 in the last).  The lengths, which would tell the last
  // row of these from the first, are on the device.
  const int64_t most = static_cast<int64_t>(max_new > 0 && max_new < ctx->rows ? max_new : ctx->rows) * p.group;
  cudaError_t e;
  if (most > 32) {
    p.min_tiles = 1;
    e = launch_attention_tiles(dim, tmK, tmV, p, ws.tiles_grid, cs);
  } else {
    // A CTA that takes fewer pages than it has warps costs more in the joining
    // than it saves: 1 / 4 / 8 / 16 / 32 pages at least take 16.0 / 15.0 / 11.9 /
    // 12.7 / 15.1 us for one token over 4096 (4 kv heads x 128).
    p.min_tiles = 8;
    e = dim == 128 ? launch_rows<128>(tmK, tmV, p, most <= 8, ws, cs) : launch_rows<64>(tmK, tmV, p, most <= 8, ws, cs);
  }
  return cuda_ok(e, "context attention launch") ? DG_OK : DG_ERR_CUDA;
}

}  // extern "C"
