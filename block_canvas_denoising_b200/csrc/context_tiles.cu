// context_tiles.cu -- attention over the 8-bit paged cache for many rows per
// kv head (canvases, prompts), on the 5th-generation tensor cores.
//
// A CTA works on 256 packed query rows (two groups of 128) by 64 keys (a
// page).  Per tile and group:
//   S = Q K^T   tcgen05.mma kind::f8f6f4, K's codes as the cache holds them
//               and Q as two E4M3 terms q = (q1 + q2) 2^-e per row, which
//               is exact for every element down to 2^-9 of the row's largest
//               (below that, off by at most 2^-17 of it); two terms at the
//               E4M3 rate cost what one bf16 product would, without a copy
//               of K in 16 bits;
//   P           one thread per row: running maximum, weights 2^(x + e - m +
//               kWeightLog2) in float16 written over S in tensor memory;
//   O += P V    tcgen05.mma kind::f16 with P from tensor memory and V's codes
//               widened to float16 (exact) by four warps of their own.
// The running maximum only moves when it is exceeded by more than 2^8, so
// O is seldom rescaled; weights stay below 2^(kWeightLog2 + 8) = 2^14.
// Measured (22 heads over 2 kv heads x 128): 32 canvases of 256 rows over 2816
// to 5376 tokens in 380 us, 960 TFLOP/s at 1.9 GHz (under a sustained load, at
// the power limit, 437 us), a canvas over 4352 in 33 us; 16 heads over 4, a canvas
// at the end of 131072 tokens, in 264 us, 1.04 PFLOP/s.  A tile takes some
// 1900 cycles, in which the tensor pipe is busy for 63 %, the special function
// unit for 38 and the issue slots for 48: what bounds it is the chain of one
// row's softmax from tensor memory to tensor memory, with two warps a scheduler
// to cover it.  An item costs some 6 tiles more, for its queries
// (2000 cycles of copies, 3600 of conversions), result (4000, L2 writes of the
// parts).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "context.h"
#include "context_attention.h"
#include "dg_internal.h"
#include "per_device.h"

namespace dg {

namespace {

constexpr int kGroupRows = 128;
constexpr int kTilesM = 2 * kGroupRows;
// Keys per tile.  Tensor memory has 256 columns for a group: O takes 128 (at
// dim 128), so S has 128, and P lies over S.  With tiles of 128 keys the next
// S has to wait for P V of this one, and products and softmax take turns
// (measured: 6200 cycles for 256 rows x 128 keys); two S of 64 keys each let
// the next product run under this tile's softmax, at the price of a Q operand
// that is read twice as often.
constexpr int kTilesN = DG_PAGE;
constexpr float kWeightLog2 = 6.f;
// Of a row's 32 pairs of weights, so many are exponentials by polynomial: the
// special function unit gives 4 a cycle and scheduler, which is half of a
// tile's time.  0 / 6 / 10 / 14 pairs: 277 / 267 / 275 / 281 us for a canvas
// over 131072 tokens.
constexpr int kPolyPairs = 6;
constexpr float kLazyLog2 = 8.f;      // the maximum may be exceeded by 2^8 before it moves
constexpr float kLargeLog2 = 4194304.f;  // 2^22

// Warp roles.  Tensor memory is read by lane quarter (warp % 4), so each
// softmax group is four consecutive warps.  Each group has an issuing warp of
// its own: one thread serving both had to poll their barriers, and was late
// for each by the time the other took.
constexpr int kMmaWarp0 = 0, kLoadWarp = 2, kPlanWarp = 3;  // issuing warps 0 and 1
constexpr int kSoftWarp0 = 4, kConvWarp0 = 12;
constexpr int kTilesThreads = 512;

constexpr int kScaleSlots = 16;  // tiles whose page scales are kept
constexpr int kPieceSlots = 8;   // pieces of work known ahead; the groups are at most kKStages tiles apart

template <int kDim>
struct TilesCfg {
  static constexpr int kRow = kDim;                             // bytes of a row of codes
  static constexpr int kQBytes = kGroupRows * kRow;             // one term of one group
  static constexpr int kKBytes = kTilesN * kRow;
  static constexpr int kVhBytes = kTilesN * kDim * 2;
  static constexpr int kKStages = 6, kV8Stages = 4, kVhStages = 4;
  static constexpr int kOffK = 4 * kQBytes;
  static constexpr int kOffV8 = kOffK + kKStages * kKBytes;
  static constexpr int kOffVh = kOffV8 + kV8Stages * kKBytes;
  static constexpr int kSmem = kOffVh + kVhStages * kVhBytes + 1024;
  static constexpr int kPartFloats = kTilesM * (kDim + 2);
  static_assert(kKStages < kPieceSlots && kKStages < kScaleSlots - 2, "slots are written before they are read");
  static_assert(kSmem <= 220 * 1024, "attention tiles exceed the shared memory of an SM");
};

// One piece of a CTA's work: some key tiles of one item.
struct Piece {
  int r, row0, nq, len, causal, mt, h;
  int tile0, tiles;     // key tiles
  int groups;           // 1 or 2 groups have rows
  int whole, c0, parts; // the whole item, or the split it belongs to
  int last;             // no piece: the end
};

struct TilesShared {
  int64_t before[DG_MAX_B + 1];
  Piece piece[kPieceSlots];
  float2 scale[kScaleSlots];  // (k scale, value exponent) of the tile's page; k scale < 0: page not there
  uint64_t k_full[6], k_empty[6], v8_full[4], v8_empty[4], vh_full[4], vh_empty[4];
  // [group], [group][S buffer].  A wait names a phase by its parity, so a
  // barrier must never be two phases from the one waited for: the last P V and
  // the one before it may both be under way, hence one o_done per buffer.
  uint64_t q_full[2], s_full[2][2], p_full[2][2], o_done[2][2];
  uint64_t sc_full[kScaleSlots], piece_full[kPieceSlots], piece_empty[kPieceSlots];
  uint32_t tmem;
};

// ---- tcgen05 for a CTA on its own -----------------------------------------
DG_DEV void tmem_alloc1(uint32_t dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
}
DG_DEV void tmem_relinquish1() { asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory"); }
DG_DEV void tmem_dealloc1(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
DG_DEV void tc_commit1(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// The descriptors come as two 32-bit halves, the low one carrying the start
// address: stepping along K or to another stage is then one 32-bit add of a
// constant.  The issuing thread has 64 cycles per instruction; with 64-bit
// descriptors put together on the spot it took 140 to 200.
// D[tmem] (+)= A[smem] B[smem]^T, E4M3, both K-major (K = 32).
DG_DEV void mma_e4m3_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem], float16 (K = 16).
DG_DEV void mma_f16_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 32 consecutive 32-bit columns of this thread's tensor-memory lane.
DG_DEV void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
// Wait for this thread's loads; the registers pass through, so that nothing
// that uses them moves ahead of the wait.
DG_DEV void tmem_ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
// The same for 16 columns, and their stores.
DG_DEV void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(addr)
               : "memory");
}
DG_DEV void tmem_ld_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
DG_DEV void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}
DG_DEV void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
               : "memory");
}
DG_DEV void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// mbarrier tests without the suspend hint: half the latency of the hinted
// form when the phase is already over (48 cycles against 84), which is what a
// chain of short waits on one path pays.
DG_DEV uint32_t mbar_over(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok;
}
// Wait for both phases (the same barrier twice for one), for at most limit_ns.
DG_DEV bool wait_over(uint32_t bar_a, uint32_t par_a, uint32_t bar_b, uint32_t par_b, uint64_t limit_ns) {
  if (mbar_over(bar_a, par_a) & mbar_over(bar_b, par_b)) return true;
  const uint64_t t0 = global_timer_ns();
#pragma unroll 1
  for (uint32_t i = 1;; ++i) {
    if (mbar_over(bar_a, par_a) & mbar_over(bar_b, par_b)) return true;
    if ((i & 63u) == 0 && global_timer_ns() - t0 > limit_ns) return false;
  }
}
DG_DEV bool wait_over(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  if (mbar_over(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
#pragma unroll 1
  for (uint32_t i = 1;; ++i) {
    if (mbar_over(bar, parity)) return true;
    if ((i & 63u) == 0 && global_timer_ns() - t0 > limit_ns) return false;
  }
}

// Descriptor of a K-major tile whose rows are one swizzle span (128 or 64
// bytes), 8-row groups one after another.
template <int kRow>
DG_DEV uint64_t desc_k_major(uint32_t saddr) {
  uint64_t d = (saddr & 0x3FFFFu) >> 4;
  d |= static_cast<uint64_t>(1u) << 16;
  d |= static_cast<uint64_t>((8 * kRow) >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(kRow == 128 ? 2u : 4u) << 61;
  return d;
}
// Descriptor of an MN-major float16 tile in the 128-byte swizzle: rows are
// keys (K), 64 elements of the head (N) each; 8-key groups 1024 bytes apart
// (stride), the next 64 elements kTilesN rows further (leading).
DG_DEV uint64_t desc_mn_major(uint32_t saddr) {
  uint64_t d = (saddr & 0x3FFFFu) >> 4;
  d |= static_cast<uint64_t>((kTilesN * 128) >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}
// kind::f16, A and B float16 (format 0), f32 accumulator, B MN-major (bit 16).
__host__ __device__ constexpr uint32_t idesc_f16_bmn(int M, int N) {
  return (1u << 4) | (1u << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Two float16 to E4M3, to nearest even, saturating.
DG_DEV uint32_t half2_to_e4m3x2(uint32_t v) {
  uint32_t d;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f16x2 t, %1;\n\tcvt.u32.u16 %0, t;\n\t}" : "=r"(d) : "r"(v));
  return d;
}
DG_DEV uint32_t sub_half2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
DG_DEV uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
DG_DEV uint32_t e4m3x2_to_half2(uint32_t w) {  // low 16 bits
  uint32_t d;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(d) : "r"(w));
  return d;
}
DG_DEV uint32_t pack_half2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Two float32 lanes in one 64-bit register pair.
DG_DEV uint64_t pack2(float x, float y) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
DG_DEV void unpack2(uint64_t v, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
DG_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
DG_DEV uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// 2^x of two numbers up to 127 without the special function unit: the
// nearest whole number n by adding 1.5 * 2^23, 2^(x - n) by the polynomial of
// degree 4 with the least largest relative error on [-1/2, 1/2] (2.6e-6, found
// by Remez exchange), n into the exponent.
// Anything below, -inf too, gives about 2^-126: nothing in float16, and next to
// nothing in a sum.  So does NaN.
DG_DEV void exp2_poly2(uint64_t v, float& x, float& y) {
  float a, b;
  unpack2(v, a, b);
  const uint64_t w = pack2(fmaxf(a, -126.f), fmaxf(b, -126.f));
  const uint64_t magic = pack2(12582912.f, 12582912.f), minus = pack2(-12582912.f, -12582912.f);
  const uint64_t t = add2(w, magic);
  const uint64_t f = fma2(add2(t, minus), pack2(-1.f, -1.f), w);
  uint64_t q = fma2(f, pack2(0.009570102207362652f, 0.009570102207362652f), pack2(0.05591785907745361f, 0.05591785907745361f));
  q = fma2(q, f, pack2(0.240247443318367f, 0.240247443318367f));
  q = fma2(q, f, pack2(0.6931217908859253f, 0.6931217908859253f));
  q = fma2(q, f, pack2(0.9999992847442627f, 0.9999992847442627f));
  float qa, qb, ta, tb;
  unpack2(q, qa, qb);
  unpack2(t, ta, tb);
  x = __uint_as_float(__float_as_uint(qa) + (__float_as_uint(ta) << 23));
  y = __uint_as_float(__float_as_uint(qb) + (__float_as_uint(tb) << 23));
}
DG_DEV float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
DG_DEV float max_of_32(const uint32_t (&u)[32]) {
  float m[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) m[k] = fmaxf(__uint_as_float(u[k]), __uint_as_float(u[28 + k]));
#pragma unroll
  for (int i = 4; i < 28; i += 8) {
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = max3(m[k], __uint_as_float(u[i + 2 * k]), __uint_as_float(u[i + 2 * k + 1]));
  }
  return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}

// A row that saw no key: its maximum never moved.  (A row of NaN that saw one
// has not moved it either, but its sum is NaN.)
DG_DEV bool saw_nothing(float m, float l) { return m == -FLT_MAX && l < 1.f; }

// A row's place in the batch.
struct Row {
  bool live;
  int lo, hi;            // keys it sees
  int64_t token, head;   // row of the batch, query head
};
DG_DEV Row row_of(const AttnParams& p, const Piece& w, int row) {
  const uint32_t rho = static_cast<uint32_t>(w.mt) * kTilesM + row;  // rows * group is below 2^31
  const int i = static_cast<int>(rho / static_cast<uint32_t>(p.group));
  Row o;
  o.live = i < w.nq;
  o.token = w.row0 + i;
  o.head = w.h * p.group + static_cast<int>(rho - i * p.group);
  Request q;
  q.nq = w.nq;
  q.len = w.len;
  q.causal = w.causal != 0;
  o.lo = o.live ? key_lo(p, q, i) : 1;
  o.hi = o.live ? key_hi(q, i) : 0;
  return o;
}

// A warp's 32 query rows (from packed row rho0 of the piece) as two E4M3
// terms in shared memory (K-major, swizzled).  The bf16 rows come by
// asynchronous copies, dim / 8 neighbouring lanes to a row, into the very
// place of the two terms -- a row of bf16 is as long as both -- and every
// thread then turns its own row: 16 reads in flight a lane and no shuffles.
// Returns the factor that turns a dot product of the thread's row into a
// logit in units of log2; NaN for a row that is not finite.
template <int kDim>
DG_DEV float prepare_q(const AttnParams& p, const Piece& w, uint32_t rho0, uint8_t* q1, uint8_t* q2, int row0) {
  constexpr int kLanes = kDim / 8;           // lanes per row
  constexpr int kAtOnce = 32 / kLanes;       // rows per step
  const int lane = threadIdx.x & 31, sub = lane / kLanes, c = lane % kLanes;
  // chunk i of a row: the first dim / 16 lie in q1, the others in q2 (a copied
  // line of 128 bytes stays one: with chunks in q1 and q2 by turns the copies
  // took twice as long)
  auto place = [&](int row, int i) {
    const int k = i & (kDim / 16 - 1);
    return (i < kDim / 16 ? q1 : q2) + (kDim == 128 ? row * 128 + ((k ^ (row & 7)) << 4) : row * 64 + ((k ^ ((row >> 1) & 3)) << 4));
  };
  // this lane's first row, and the steps to its next ones, without a division
  const uint32_t group = static_cast<uint32_t>(p.group);
  uint32_t i = (rho0 + sub) / group, g = rho0 + sub - i * group;  // query row and head within the kv head
  const uint8_t* src = p.q + (w.row0 + i) * p.q_row + (static_cast<int64_t>(w.h) * group + g) * p.q_head + 16 * c;
  const uint32_t step_i = kAtOnce / group, step_g = kAtOnce - step_i * group;
  const int64_t step = step_i * p.q_row + step_g * p.q_head, turn = p.q_row - group * p.q_head;
#pragma unroll
  for (int k = 0; k < 32 / kAtOnce; ++k) {
    // a row that is not there: nothing is read and the place is filled with zeros
    const bool live = static_cast<int>(i) < w.nq;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(place(row0 + k * kAtOnce + sub, c))),
                 "l"(live ? src : p.q), "r"(live ? 16 : 0)
                 : "memory");
    i += step_i;
    g += step_g;
    src += step;
    if (g >= group) {
      g -= group;
      ++i;
      src += turn;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  const int row = row0 + lane;
  // The largest magnitude, two bf16 at a time (a NaN passes through): its
  // exponent, all ones if something is not finite.
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < kDim / 8; ++i) {
    const uint4 v = *reinterpret_cast<const uint4*>(place(row, i));
    most = max_bf16x2(max_bf16x2(most, max_bf16x2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu)),
                      max_bf16x2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
  }
  const uint32_t top = max(most << 16, most & 0xFFFF0000u);  // float32 bits
  const int b = static_cast<int>(top >> 23);
  const int e = b == 0 ? 0 : min(7 - (b - 127), 120);  // largest magnitude to [2^7, 2^8)
  const bool finite = b < 255;
  const float f = pow2i(e);
  // Chunks 2i and 2i + 1 become chunk i of both terms, in an order in which
  // every place has been read before it is written; a quarter of the row waits
  // in registers.
  auto terms = [&](int i, const uint4& v0, const uint4& v1) {
    const uint32_t u[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    uint32_t t1[4], t2[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // float16 holds the scaled values to 2^-25, far below what the terms do
      const uint32_t x0 = pack_half2(__uint_as_float(u[2 * j] << 16) * f, __uint_as_float(u[2 * j] & 0xFFFF0000u) * f);
      const uint32_t x1 = pack_half2(__uint_as_float(u[2 * j + 1] << 16) * f, __uint_as_float(u[2 * j + 1] & 0xFFFF0000u) * f);
      const uint32_t lo = half2_to_e4m3x2(x0), hi = half2_to_e4m3x2(x1);
      t1[j] = finite ? (lo | hi << 16) : 0x7F7F7F7Fu;  // a row that is not finite: NaN throughout
      t2[j] = half2_to_e4m3x2(sub_half2(x0, e4m3x2_to_half2(lo))) | half2_to_e4m3x2(sub_half2(x1, e4m3x2_to_half2(hi))) << 16;
    }
    *reinterpret_cast<uint4*>(place(row, i)) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
    *reinterpret_cast<uint4*>(place(row, kDim / 16 + i)) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
  };
  auto chunk = [&](int i) { return *reinterpret_cast<const uint4*>(place(row, i)); };
  constexpr int kH = kDim / 32;
  uint4 kept[kH];  // chunks kH .. 2 kH - 1
#pragma unroll
  for (int j = 0; j < kH; ++j) kept[j] = chunk(kH + j);
#pragma unroll 2
  for (int i = 2 * kH - 1; i >= kH; --i) terms(i, chunk(2 * i), chunk(2 * i + 1));
#pragma unroll
  for (int i = 0; i < kH / 2; ++i) terms(i, chunk(2 * i), chunk(2 * i + 1));
#pragma unroll
  for (int i = kH / 2; i < kH; ++i) terms(i, kept[2 * i - kH], kept[2 * i + 1 - kH]);
  return finite ? p.scale_log2 * pow2i(-e) : __int_as_float(0x7fc00000);
}

template <int kDim>
__global__ void __launch_bounds__(kTilesThreads, 1)
attention_tiles_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const __grid_constant__ AttnParams p) {
  using Cfg = TilesCfg<kDim>;
  using S = Split<kTilesM, kTilesN, 6>;  // queries and result of an item take as long as some 6 tiles
  extern __shared__ uint8_t smem_raw[];
  __shared__ TilesShared sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::kKStages; ++s) {
      mbar_init(smem_u32(&sh.k_full[s]), 1);
      mbar_init(smem_u32(&sh.k_empty[s]), 2);
    }
    for (int s = 0; s < Cfg::kV8Stages; ++s) {
      mbar_init(smem_u32(&sh.v8_full[s]), 1);
      mbar_init(smem_u32(&sh.v8_empty[s]), 4);
    }
    for (int s = 0; s < Cfg::kVhStages; ++s) {
      mbar_init(smem_u32(&sh.vh_full[s]), 4);
      mbar_init(smem_u32(&sh.vh_empty[s]), 2);
    }
    for (int s = 0; s < kPieceSlots; ++s) {
      mbar_init(smem_u32(&sh.piece_full[s]), 1);
      mbar_init(smem_u32(&sh.piece_empty[s]), 15);  // 2 issuing warps, loader, 4 converter and 8 softmax warps
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_u32(&sh.q_full[s]), 4);
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_u32(&sh.s_full[s][b]), 1);
        mbar_init(smem_u32(&sh.p_full[s][b]), 4);
        mbar_init(smem_u32(&sh.o_done[s][b]), 1);
      }
    }
    for (int s = 0; s < kScaleSlots; ++s) mbar_init(smem_u32(&sh.sc_full[s]), 1);
    fence_mbarrier_init();
  }
  if (warp == kMmaWarp0) {
    tmem_alloc1(smem_u32(&sh.tmem), 512);
    tmem_relinquish1();
  }
  wait_for_previous_kernel();
  allow_next_kernel();
  S::totals(p, sh.before);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  // columns: S (and P over it) of group g, buffer b at 128 g + 64 b, O at 256 + 128 g
  const int64_t total = sh.before[p.B];
  const int64_t even = quotient(total + gridDim.x - 1, gridDim.x);
  const int64_t per = even > p.min_tiles ? even : p.min_tiles;

  bool ok = true;
  auto wait = [&](uint64_t& bar, uint32_t parity) {
    if (ok && !wait_over(smem_u32(&bar), parity, p.wait_ns)) {
      ok = false;
      atomicOr(p.err, kErrWaitContext);
    }
  };
  auto wait2 = [&](uint64_t& a, uint32_t pa, uint64_t& b, uint32_t pb) {
    if (ok && !wait_over(smem_u32(&a), pa, smem_u32(&b), pb, p.wait_ns)) {
      ok = false;
      atomicOr(p.err, kErrWaitContext);
    }
  };
  // the piece list, read by every role at its own pace
  auto next_piece = [&](int n) -> const Piece& {
    wait(sh.piece_full[n % kPieceSlots], (n / kPieceSlots) & 1);
    return sh.piece[n % kPieceSlots];
  };
  auto done_piece = [&](int n) {  // one lane per warp
    mbar_arrive(smem_u32(&sh.piece_empty[n % kPieceSlots]));
  };

  if (warp == kPlanWarp) {
    // ---- the pieces of this CTA's range, some ahead of their use
    int64_t pos = blockIdx.x * per;
    const int64_t end = min(pos + per, total);
    Piece split = {};
    for (int n = 0; ok; ++n) {
      if (n >= kPieceSlots) wait(sh.piece_empty[n % kPieceSlots], ((n / kPieceSlots) & 1) ^ 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      Piece w;
      S it;
      if (pos < end) {
        it.find(p, sh.before, pos);
        pos = max(pos, it.begin);
      }
      w.last = pos >= end;
      if (!w.last) {
        const int64_t item_end = it.begin + it.tiles;
        w.r = it.r;
        w.row0 = it.q.row0;
        w.nq = it.q.nq;
        w.len = it.q.len;
        w.causal = it.q.causal;
        w.mt = it.mt;
        w.h = it.h;
        w.tile0 = it.first + static_cast<int>(pos - it.begin);
        w.tiles = static_cast<int>(min(item_end, end) - pos);
        w.groups = static_cast<int64_t>(it.q.nq) * p.group - static_cast<int64_t>(it.mt) * kTilesM > kGroupRows ? 2 : 1;
        w.whole = w.tiles == it.tiles;
        w.c0 = static_cast<int>(quotient(it.begin, per));
        w.parts = static_cast<int>(quotient(item_end - 1, per)) - w.c0 + 1;
        pos += w.tiles;
        if (!w.whole && w.c0 == static_cast<int>(blockIdx.x)) split = w;  // an item that begins here and ends elsewhere
      }
      if (lane == 0) {
        sh.piece[n % kPieceSlots] = w;
        mbar_arrive(smem_u32(&sh.piece_full[n % kPieceSlots]));
      }
      if (w.last) break;
    }
    if (lane == 0) static_cast<Piece*>(p.splits)[blockIdx.x] = split;  // for the kernel that joins the parts
  } else if (warp == kLoadWarp) {
    // ---- copies of K and V codes, and the pages' scales
    const uint64_t policy = policy_evict_last();  // row tiles of a head share its keys
    int T = 0, issued_k = 0, issued_v = 0;
    for (int n = 0; ok; ++n) {
      const Piece& w = next_piece(n);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok || w.last) break;
      const int last_page = (w.len + DG_PAGE - 1) / DG_PAGE - 1;
      int id = 0;
      float ks = 0.f, ve = 0.f;
      for (int j = 0; j < w.tiles; ++j, ++T) {
        if ((j & 31) == 0) {  // ids and scales of the next 32 pages, one per lane
          const int pg = w.tile0 + j + lane;
          id = -1;
          if (j + lane < w.tiles && pg <= last_page && pg < p.max_pages)
            id = p.table[static_cast<size_t>(w.r) * p.max_pages + pg];
          if (id < 0 || id >= p.pages) {
            id = p.pages;  // outside the tensor: the copy fills zeros
            ks = -1.f;     // and its keys are not seen
            ve = 0.f;
          } else {
            const size_t at = static_cast<size_t>(id) * p.kv_heads + w.h;
            ks = p.k_scale[at];
            ve = static_cast<float>(static_cast<int>(__float_as_uint(p.v_scale[at]) >> 23) - 127);
          }
        }
        const int y = (__shfl_sync(0xffffffffu, id, j & 31) * p.kv_heads + w.h) * DG_PAGE;
        const float ks_j = __shfl_sync(0xffffffffu, ks, j & 31), ve_j = __shfl_sync(0xffffffffu, ve, j & 31);
        const int st = T % Cfg::kKStages, sv = T % Cfg::kV8Stages;
        wait(sh.k_empty[st], ((T / Cfg::kKStages) & 1) ^ 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          // The slot was last read for tile T - kScaleSlots.  With K stage T %
          // kKStages free, both groups have begun tile T - kKStages, and so
          // every softmax warp is past tile T - kKStages - 2.
          sh.scale[T % kScaleSlots] = make_float2(ks_j, ve_j);
          mbar_arrive(smem_u32(&sh.sc_full[T % kScaleSlots]));
          const uint32_t bar = smem_u32(&sh.k_full[st]);
          mbar_arrive_expect_tx(bar, Cfg::kKBytes);
          tma_load_2d(smem_u32(smem + Cfg::kOffK + st * Cfg::kKBytes), &tmK, bar, 0, y, policy);
        }
        issued_k = T + 1;
        wait(sh.v8_empty[sv], ((T / Cfg::kV8Stages) & 1) ^ 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t bar = smem_u32(&sh.v8_full[sv]);
          mbar_arrive_expect_tx(bar, Cfg::kKBytes);
          tma_load_2d(smem_u32(smem + Cfg::kOffV8 + sv * Cfg::kKBytes), &tmV, bar, 0, y, policy);
        }
        issued_v = T + 1;
      }
      __syncwarp();
      if (lane == 0) done_piece(n);
    }
    // every copy has landed before the CTA goes
    for (int t = max(issued_k - Cfg::kKStages, 0); t < issued_k; ++t)
      mbar_wait_bounded(smem_u32(&sh.k_full[t % Cfg::kKStages]), (t / Cfg::kKStages) & 1, p.wait_ns);
    for (int t = max(issued_v - Cfg::kV8Stages, 0); t < issued_v; ++t)
      mbar_wait_bounded(smem_u32(&sh.v8_full[t % Cfg::kV8Stages]), (t / Cfg::kV8Stages) & 1, p.wait_ns);
  } else if (warp < kMmaWarp0 + 2) {
    // ---- the issuing warps: the next tile's S = Q K^T ahead of this tile's
    // O += P V
    const int gi = warp - kMmaWarp0;
    constexpr uint32_t idesc_s = instr_desc_e4m3_f32(kGroupRows, kTilesN);
    constexpr uint32_t idesc_o = idesc_f16_bmn(kGroupRows, kDim);
    const uint64_t q0 = desc_k_major<kDim>(smem_u32(smem + 2 * gi * Cfg::kQBytes));
    const uint64_t k0 = desc_k_major<kDim>(smem_u32(smem + Cfg::kOffK)), v0 = desc_mn_major(smem_u32(smem + Cfg::kOffVh));
    const uint32_t q_lo = static_cast<uint32_t>(q0), k_lo = static_cast<uint32_t>(k0), v_lo = static_cast<uint32_t>(v0);
    const uint32_t k_hi = static_cast<uint32_t>(k0 >> 32), v_hi = static_cast<uint32_t>(v0 >> 32);
    const uint32_t t_s = tmem + 128 * gi, t_o = tmem + 256 + 128 * gi;
    uint32_t sk = 0, pk = 0, sv = 0, pv = 0;
    uint32_t a = 0, b = 0;  // products S and P V issued so far (mod 2^32)
    uint32_t pieces = 0;
    for (int n = 0; ok && lane == 0; ++n) {
      const Piece& w = next_piece(n);
      if (!ok || w.last) break;
      const int tiles = w.tiles;
      const bool on = gi < w.groups;
      auto score = [&](bool first) {
        // The buffer is free once P V of two tiles back is done.  A piece's
        // first S comes after the last P V before it, any other ahead of the P V
        // in between.
        if (on && first) wait(sh.q_full[gi], pieces & 1);
        const uint32_t behind = first ? b - 1 : a - 2;
        if (on && static_cast<int>(behind) >= 0)
          wait2(sh.k_full[sk], pk, sh.o_done[gi][behind & 1], (behind >> 1) & 1);
        else
          wait(sh.k_full[sk], pk);
        if (!ok) return;
        if (on) {
          tc_fence_after();
          const uint32_t kb = k_lo + sk * (Cfg::kKBytes >> 4), d = t_s + 64 * (a & 1);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int k = 0; k < kDim / 32; ++k)
              mma_e4m3_ss(d, q_lo + t * (Cfg::kQBytes >> 4) + 2 * k, k_hi, kb + 2 * k, k_hi, idesc_s, t + k > 0);
          }
          tc_commit1(smem_u32(&sh.s_full[gi][a & 1]));
          tc_commit1(smem_u32(&sh.k_empty[sk]));
          ++a;
        } else {
          mbar_arrive(smem_u32(&sh.k_empty[sk]));
        }
        if (++sk == Cfg::kKStages) {
          sk = 0;
          pk ^= 1;
        }
      };
      score(true);
      for (int j = 0; j < tiles && ok; ++j) {
        if (j + 1 < tiles) score(false);
        if (on)
          wait2(sh.p_full[gi][b & 1], (b >> 1) & 1, sh.vh_full[sv], pv);
        else
          wait(sh.vh_full[sv], pv);
        if (!ok) break;
        if (on) {
          tc_fence_after();
          const uint32_t vb = v_lo + sv * (Cfg::kVhBytes >> 4), s = t_s + 64 * (b & 1);
          mma_f16_ts(t_o, s, vb, v_hi, idesc_o, j > 0);
#pragma unroll
          for (int k = 1; k < kTilesN / 16; ++k) mma_f16_ts(t_o, s + 8 * k, vb + 128 * k, v_hi, idesc_o, 1u);
          tc_commit1(smem_u32(&sh.o_done[gi][b & 1]));
          tc_commit1(smem_u32(&sh.vh_empty[sv]));
          ++b;
        } else {
          mbar_arrive(smem_u32(&sh.vh_empty[sv]));
        }
        if (++sv == Cfg::kVhStages) {
          sv = 0;
          pv ^= 1;
        }
      }
      if (on) ++pieces;
      if (ok) done_piece(n);
    }
    // its products have completed before tensor memory is freed
    if (a > b) mbar_wait_bounded(smem_u32(&sh.s_full[gi][(a - 1) & 1]), ((a - 1) >> 1) & 1, p.wait_ns);
    if (b > 0) mbar_wait_bounded(smem_u32(&sh.o_done[gi][(b - 1) & 1]), ((b - 1) >> 1) & 1, p.wait_ns);
    __syncwarp();
  } else if (warp >= kConvWarp0) {
    // ---- V's codes to float16: half a key per thread; both layouts keep a key's
    // row together and swizzle its 16-byte chunks by the row, so eight
    // threads read and write all banks
    const int tid = threadIdx.x - kConvWarp0 * 32, key = tid & 63, side = tid >> 6;
    int T = 0;
    for (int n = 0; ok; ++n) {
      const Piece& w = next_piece(n);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok || w.last) break;
      const int tile0 = w.tile0, tiles = w.tiles, len = w.len;
      for (int j = 0; j < tiles && ok; ++j, ++T) {
        const int sv = T % Cfg::kV8Stages, so = T % Cfg::kVhStages;
        wait(sh.v8_full[sv], (T / Cfg::kV8Stages) & 1);
        wait(sh.vh_empty[so], ((T / Cfg::kVhStages) & 1) ^ 1);
        const uint8_t* src = smem + Cfg::kOffV8 + sv * Cfg::kKBytes + key * Cfg::kRow;
        uint8_t* dst = smem + Cfg::kOffVh + so * Cfg::kVhBytes + key * 128;
        const bool there = (tile0 + j) * kTilesN + key < len;  // behind the last token: zeros, whatever is there
#pragma unroll
        for (int i = 0; i < kDim / 32; ++i) {
          const int c = side * (kDim / 32) + i;
          const int at = kDim == 128 ? (c ^ (key & 7)) << 4 : (c ^ ((key >> 1) & 3)) << 4;
          uint4 v = *reinterpret_cast<const uint4*>(src + at);
          if (!there) v = make_uint4(0, 0, 0, 0);
          const uint4 lo = make_uint4(e4m3x2_to_half2(v.x), e4m3x2_to_half2(v.x >> 16), e4m3x2_to_half2(v.y), e4m3x2_to_half2(v.y >> 16));
          const uint4 hi = make_uint4(e4m3x2_to_half2(v.z), e4m3x2_to_half2(v.z >> 16), e4m3x2_to_half2(v.w), e4m3x2_to_half2(v.w >> 16));
          uint8_t* d = dst + (c >> 2) * (kTilesN * 128);
          const int o = 2 * (c & 3);
          *reinterpret_cast<uint4*>(d + ((o ^ (key & 7)) << 4)) = lo;
          *reinterpret_cast<uint4*>(d + (((o + 1) ^ (key & 7)) << 4)) = hi;
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&sh.vh_full[so]));
          mbar_arrive(smem_u32(&sh.v8_empty[sv]));
        }
      }
      __syncwarp();
      if (lane == 0) done_piece(n);
    }
  } else {
    // ---- softmax: one thread per row
    const int gi = (warp - kSoftWarp0) >> 2;
    const int quarter = warp & 3;
    const int row = gi * kGroupRows + quarter * 32 + lane;   // of the item
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tmem + lanes + 128 * gi, t_o = tmem + lanes + 256 + 128 * gi;
    uint8_t* q1 = smem + 2 * gi * Cfg::kQBytes;
    uint8_t* q2 = q1 + Cfg::kQBytes;
    int T = 0, used = 0;
    float fac = 0.f;
    int key_first = 1, key_last = 0;  // the keys this thread's row sees
    auto begin_piece = [&](const Piece& w) {
      const Row o = row_of(p, w, row);
      // a row that is not there (its query is 0, its result goes nowhere)
      // counts as seeing everything, so that it asks for no masks
      key_first = o.live ? o.lo : 0;
      key_last = o.live ? o.hi : 0x7FFFFFF0;
      fac = prepare_q<kDim>(p, w, w.mt * kTilesM + gi * kGroupRows + quarter * 32, q1, q2, quarter * 32);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.q_full[gi]));
    };
    // Round n works on piece n, prepares the queries of piece n + 1 and writes
    // the result of piece n; round -1 prepares only.  One place in the code
    // for each: what runs once per piece runs from a cold instruction cache,
    // and costs by its length.
    for (int n = -1;; ++n) {
      const Piece& w = n < 0 ? next_piece(0) : next_piece(n);  // in shared memory until done_piece
      ok = __all_sync(0xffffffffu, ok);
      if (!ok || w.last) break;
      const bool on = n >= 0 && gi < w.groups;
      const int tile0 = w.tile0, tiles = n < 0 ? 0 : w.tiles;
      float m = -FLT_MAX, l = 0.f;
      if (!on) {
        T += tiles;
      } else {
        // Tiles [full0, full1) are seen whole by every row of the warp.
        int full0 = (key_first + kTilesN - 1) / kTilesN - tile0, full1 = (key_last + 1) / kTilesN - tile0;
        if (key_last < key_first) full1 = -1;
        full0 = __reduce_max_sync(0xffffffffu, full0);
        full1 = __reduce_min_sync(0xffffffffu, full1);
        wait(sh.s_full[gi][used & 1], (used >> 1) & 1);  // before scales: this warp may have skipped tiles
        wait(sh.sc_full[T % kScaleSlots], (T / kScaleSlots) & 1);
        float2 sc = sh.scale[T % kScaleSlots];
        for (int j = 0; j < tiles; ++j) {
          const uint32_t t_p = t_s + 64 * (used & 1);
          if (j > 0) wait(sh.s_full[gi][used & 1], (used >> 1) & 1);
          tc_fence_after();
          uint32_t u[2][32];
          tmem_ld32(t_p, u[0]);
          tmem_ld_wait(u[0]);
          tmem_ld32(t_p + 32, u[1]);
          float top = max_of_32(u[0]);
          tmem_ld_wait(u[1]);
          if (j < full0 || j >= full1 || !(sc.x > 0.f)) {
            const int lo = key_first - (tile0 + j) * kTilesN, span = sc.x > 0.f ? key_last - key_first : -1;
#pragma unroll
            for (int i = 0; i < kTilesN; ++i) {
              const bool seen = span >= 0 && static_cast<uint32_t>(i - lo) <= static_cast<uint32_t>(span);
              u[i / 32][i % 32] = seen ? u[i / 32][i % 32] : 0xFF800000u;
            }
            top = max_of_32(u[0]);
          }
          top = fmaxf(top, max_of_32(u[1]));
          float s[kTilesN];
#pragma unroll
          for (int i = 0; i < kTilesN; ++i) s[i] = __uint_as_float(u[i / 32][i % 32]);
          float c = fmaxf(fac * fabsf(sc.x), FLT_MIN);
          top = __fmul_rn(top, c) + sc.y;
          if (__any_sync(0xffffffffu, top > m + kLazyLog2 || fabsf(top) > kLargeLog2)) {
            // The weights take s c - m in one fused step, m being the rounded
            // maximum: a difference that is off by up to 2^-24 |m|, the same
            // for the whole row, and so of no effect until it nears the
            // weights' headroom.  Logits that large are rounded first, and the
            // maximum then follows them closely.
            const bool large = __any_sync(0xffffffffu, fabsf(top) > kLargeLog2 && top > -INFINITY);
            if (large) {
#pragma unroll
              for (int i = 0; i < kTilesN; ++i) s[i] *= c;
              c = 1.f;
            }
            const float mn = top > m + (large ? 0.f : kLazyLog2) ? top : m;
            const float shrink = exp2f(m - mn);
            m = mn;
            l *= shrink;
            if (j > 0 && __any_sync(0xffffffffu, shrink != 1.f)) {  // O holds the tiles before; their last product has to be done
              wait(sh.o_done[gi][(used - 1) & 1], ((used - 1) >> 1) & 1);
              tc_fence_after();
#pragma unroll 1
              for (int c16 = 0; c16 < kDim / 16; ++c16) {
                uint32_t x[16];
                tmem_ld16(t_o + 16 * c16, x);
                tmem_ld_wait(x);
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * shrink);
                tmem_st16(t_o + 16 * c16, x);
              }
            }
          }
          const uint64_t cc = pack2(c, c);
          const float off = sc.y - m + kWeightLog2;
          const uint64_t bb = pack2(off, off);
          uint64_t sum[4] = {0, 0, 0, 0};
          uint32_t h[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float x, y;
            const uint64_t v = fma2(pack2(s[2 * i], s[2 * i + 1]), cc, bb);
            if ((i * kPolyPairs) / 32 != ((i + 1) * kPolyPairs) / 32) {
              exp2_poly2(v, x, y);
            } else {
              unpack2(v, x, y);
              x = exp2_fast(x);
              y = exp2_fast(y);
            }
            sum[i & 3] = add2(sum[i & 3], pack2(x, y));
            h[i] = pack_half2(x, y);
          }
          tmem_st32(t_p, h);
          // while the weights are on their way: the row's sum, the next scales
          float x, y;
          unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), x, y);
          l += (x + y) * pow2i(-static_cast<int>(sc.y));
          // A row that is not finite: NaN as soon as it sees a key.  Its weights
          // do not say so, since those by polynomial are numbers.
          if (fac != fac) {
            const int key0 = (tile0 + j) * kTilesN;
            if (sc.x > 0.f && max(key_first, key0) <= min(key_last, key0 + kTilesN - 1)) l = fac;
          }
          ++T;
          if (j + 1 < tiles) {  // there long since
            wait(sh.sc_full[T % kScaleSlots], (T / kScaleSlots) & 1);
            sc = sh.scale[T % kScaleSlots];
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sh.p_full[gi][used & 1]));
          ++used;
        }
      }
      // the next piece's queries, so that its first product runs while this
      // piece's result is written
      {
        const Piece& next = next_piece(n + 1);
        if (ok && !next.last && gi < next.groups) begin_piece(next);
      }
      if (n < 0) continue;
      const Row mine = row_of(p, w, row);
      const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (static_cast<int>(blockIdx.x) == w.c0 ? 1 : 0);
      auto store_lse = [&](float top, float sum) {
        if (p.lse != nullptr && mine.live)
          p.lse[mine.token * (static_cast<int64_t>(p.kv_heads) * p.group) + mine.head] =
              saw_nothing(top, sum) ? -INFINITY : (top - kWeightLog2 + log2f(sum)) * kLn2;
      };
      uint8_t* dst = p.out + mine.token * p.out_row + mine.head * p.out_head;
      if (on) {
        wait(sh.o_done[gi][(used - 1) & 1], ((used - 1) >> 1) & 1);
        tc_fence_after();
        const float inv = saw_nothing(m, l) ? 0.f : 1.0f / l;
        float* part = p.part + slot * Cfg::kPartFloats;
#pragma unroll 1
        for (int c = 0; c < kDim / 32; ++c) {
          uint32_t x[32];
          tmem_ld32(t_o + 32 * c, x);
          tmem_ld_wait(x);
          if (w.whole) {
            if (mine.live) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(x[8 * k + 2 * i]) * inv,
                                                                 __uint_as_float(x[8 * k + 2 * i + 1]) * inv);
                  b[i] = *reinterpret_cast<const uint32_t*>(&v);
                }
                *reinterpret_cast<uint4*>(dst + 64 * c + 16 * k) = make_uint4(b[0], b[1], b[2], b[3]);
              }
            }
          } else {  // [dim / 4][256] float4: a warp writes 512 bytes in a row
#pragma unroll
            for (int k = 0; k < 8; ++k)
              reinterpret_cast<uint4*>(part)[(8 * c + k) * kTilesM + row] =
                  make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
          }
        }
        tc_fence_before();
        if (w.whole) {
          store_lse(m, l);
        } else {
          part[kTilesM * kDim + row] = m;
          part[kTilesM * kDim + kTilesM + row] = l;
        }
      }
      __syncwarp();
      if (lane == 0) done_piece(n);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp0) tmem_dealloc1(tmem, 512);
}

// Joins the parts of the items that more than one CTA worked on, in split
// order, so results do not depend on which CTA was done first.  Block (c, y)
// works on the item that begins in CTA c's range and ends behind it, if there
// is one; a warp on 32 rows x 8 elements, every read of eight parts before the
// first use.  For one canvas, 22 items in 7 parts of 133 KB each, spread over
// the whole device, it is the latency that counts: with 16 elements and four
// parts at once the canvas takes 34.8 instead of 33.1 us, while 32 canvases,
// whose items have two parts, take 381 instead of 383 (one CTA joining an item
// alone took 32 us).
constexpr int kJoinThreads = 256;
constexpr int kJoinParts = 8, kJoinVec = 2;  // parts at once, float4 of each
template <int kDim>
__global__ void __launch_bounds__(kJoinThreads)
attention_join_kernel(const __grid_constant__ AttnParams p) {
  wait_for_previous_kernel();
  allow_next_kernel();
  constexpr int kPartFloats = TilesCfg<kDim>::kPartFloats;
  const Piece w = static_cast<const Piece*>(p.splits)[blockIdx.x];
  if (w.parts < 2) return;
  const int unit = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int row = (unit & 7) * 32 + lane, c = unit >> 3;  // elements from 4 kJoinVec c
  if (c >= kDim / (4 * kJoinVec)) return;
  const Row o = row_of(p, w, row);
  if (!o.live) return;
  auto part_of = [&](int i) { return p.part + static_cast<size_t>(2 * (w.c0 + i) + (i == 0 ? 1 : 0)) * kPartFloats; };
  float top = -FLT_MAX, sum = 0.f, x[4 * kJoinVec] = {};
  for (int i0 = 0; i0 < w.parts; i0 += kJoinParts) {  // every read of some parts before the first use
    float m[kJoinParts], l[kJoinParts];
    float4 v[kJoinParts][kJoinVec];
#pragma unroll
    for (int i = 0; i < kJoinParts; ++i) {
      const float* src = part_of(min(i0 + i, w.parts - 1));
      m[i] = i0 + i < w.parts ? __ldcg(src + kTilesM * kDim + row) : -FLT_MAX;
      l[i] = i0 + i < w.parts ? __ldcg(src + kTilesM * kDim + kTilesM + row) : 0.f;
#pragma unroll
      for (int k = 0; k < kJoinVec; ++k)
        v[i][k] = i0 + i < w.parts ? __ldcg(reinterpret_cast<const float4*>(src) + (kJoinVec * c + k) * kTilesM + row)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float now = top;
#pragma unroll
    for (int i = 0; i < kJoinParts; ++i) now = fmaxf(now, m[i]);
    const float old = join_weight(top, now);
    top = now;
    sum *= old;
#pragma unroll
    for (int k = 0; k < 4 * kJoinVec; ++k) x[k] *= old;
#pragma unroll
    for (int i = 0; i < kJoinParts; ++i) {
      const float f = join_weight(m[i], top);
      sum += l[i] * f;
#pragma unroll
      for (int k = 0; k < kJoinVec; ++k) {
        x[4 * k] += v[i][k].x * f;
        x[4 * k + 1] += v[i][k].y * f;
        x[4 * k + 2] += v[i][k].z * f;
        x[4 * k + 3] += v[i][k].w * f;
      }
    }
  }
  const float inv = saw_nothing(top, sum) ? 0.f : 1.0f / sum;
  uint32_t b[2 * kJoinVec];
#pragma unroll
  for (int i = 0; i < 2 * kJoinVec; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i] * inv, x[2 * i + 1] * inv);
    b[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  uint4* dst = reinterpret_cast<uint4*>(p.out + o.token * p.out_row + o.head * p.out_head + 8 * kJoinVec * c);
#pragma unroll
  for (int k = 0; k < kJoinVec / 2; ++k) dst[k] = make_uint4(b[4 * k], b[4 * k + 1], b[4 * k + 2], b[4 * k + 3]);
  if (p.lse != nullptr && c == 0)
    p.lse[o.token * (static_cast<int64_t>(p.kv_heads) * p.group) + o.head] =
        saw_nothing(top, sum) ? -INFINITY : (top - kWeightLog2 + log2f(sum)) * kLn2;
}

template <int kDim>
int grid_of() {
  static PerDevice<int> cache;
  int dev = -1, n = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  const bool got = cache.get(dev, [](int* v) {
    if (cudaFuncSetAttribute(attention_tiles_kernel<kDim>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             TilesCfg<kDim>::kSmem) != cudaSuccess)
      return false;
    int per_sm = 0;
    const int sms = device_sms();
    if (sms <= 0 || cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, attention_tiles_kernel<kDim>, kTilesThreads,
                                                                  TilesCfg<kDim>::kSmem) != cudaSuccess || per_sm < 1)
      return false;
    *v = sms;
    return true;
  }, &n);
  return got ? n : -1;
}

}  // namespace

int tiles_grid(int dim) { return dim == 128 ? grid_of<128>() : grid_of<64>(); }
size_t tiles_part_floats(int dim) { return dim == 128 ? TilesCfg<128>::kPartFloats : TilesCfg<64>::kPartFloats; }

size_t tiles_split_bytes() { return sizeof(Piece); }

namespace {
template <int kDim>
cudaError_t launch(const CUtensorMap& tmK, const CUtensorMap& tmV, const AttnParams& p, int grid, cudaStream_t stream) {
  const cudaError_t e = launch_context(attention_tiles_kernel<kDim>, dim3(grid), kTilesThreads, TilesCfg<kDim>::kSmem, stream, tmK, tmV, p);
  if (e != cudaSuccess) return e;
  return launch_context(attention_join_kernel<kDim>, dim3(grid, kDim / (4 * kJoinVec)), kJoinThreads, 0, stream, p);
}
}  // namespace

cudaError_t launch_attention_tiles(int dim, const CUtensorMap& tmK, const CUtensorMap& tmV, const AttnParams& p,
                                   int grid, cudaStream_t stream) {
  return dim == 128 ? launch<128>(tmK, tmV, p, grid, stream) : launch<64>(tmK, tmV, p, grid, stream);
}

}  // namespace dg
