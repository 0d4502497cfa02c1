// sgmv_matmul_tiled.h -- gfx950 tiled kernel of the shared projection with
// adapters and of the grouped products.  Internal to libsgmv.
//
// A workgroup computes BM rows x BN columns, C^T = W . X^T on
// v_mfma_f32_16x16x32 (weight rows are the instruction's rows, tokens its
// columns, so that a lane ends up with consecutive columns of one token).
//
// Staging.  A step of 64 along the contraction is staged in LDS as four
// halves: A0, A1 (the input rows, BM / 2 each) and B0, B1 (the weight rows,
// BN / 2 each), loaded straight from memory into LDS 16 bytes a lane, no
// registers on the way.  A half is rows of 128 bytes, eight 16-byte blocks;
// block c of row r lies in slot c ^ (r & 7), so that the eight lanes which
// the LDS serves at a time read eight different slots.  The load writes
// LDS in lane order, so each lane fetches the block that belongs into its
// slot.  Out-of-range rows and blocks (past the tile's rows, the matrix's
// columns or the contraction) read zero through the buffer's bounds.
//
// A wave owns a quarter of the tile (a half of each half).  A step's matrix
// instructions come in two parts of 32 along the contraction.  During part 1
// all operands of the next step are read into registers (three sets of a
// part's operands, rotating), so that its LDS is free half a step later and is
// refilled with the step after next, most or all of it during part 0; the loads have
// one to one and a half steps to arrive.  Evenly spread they cost least: all
// of them in the first half of part 0 is 6-8% slower.  Barriers: before part 1 (the next step has
// arrived, for every wave) and before part 0 (every wave has read it).
//
// What bounds it: with 256 x 256 tiles the matrix instructions (busy 80% of the
// compute units' time at 8192 x 8192 x 8192, 732-742 us, 1480-1501 TFLOP/s; the rest
// is barriers and the tiles' first and last steps); before loads had more
// than one step to arrive, the loads did (884 us).  Prefill of 16384 tokens,
// hidden 4096 -> 28672: 2662-2694 us = 1428-1446 TFLOP/s, with 64 adapters of
// rank 64 3002 us (segments of whole tiles; 3117-3216 of uneven lengths).  The 128 x
// 128 tile moves twice the bytes per product and wins where the large one
// leaves compute units idle (512 x 4096 x 4096: 41 us against 79) and for
// experts with few rows (64 of 96 rows: their weights at 4.4 TB/s).
//
// Microscaled 4-bit operands: a step's 128 bytes of a row are two groups of 128
// values, products are v_mfma_scale_f32_16x16x128, four times the values a
// byte and an instruction.  8192 x 8192 x 8192 takes 284 us = 3870 TFLOP/s (without its
// loads of scales 255), 16384 x 28672 x 4096 1206 us, with 64 adapters of rank 64 1520;
// a step is half as long as with 16-bit values, so that a tile's first loads
// and its stores weigh twice as much (13 of 43 us of a tile at 4096 values).  One
// workgroup a compute unit walking over tiles, the next one's loads issued ahead
// of the stores, spilled registers: 473, 1716 and 1786 us.
#pragma once

#include <type_traits>
#include <utility>

#include "sgmv_matmul.h"
#include "sgmv_mx.h"

namespace sgmv {
namespace dev {

typedef __attribute__((address_space(3))) void lds_void;

// The shape of a tiled kernel: WM x WN waves, each FM x FN blocks of 16 x 16
// per pair of halves.
template <int WM_, int WN_, int FM_, int FN_, int OCC>
struct TileShape {
  static constexpr int WM = WM_, WN = WN_, FM = FM_, FN = FN_;
  static constexpr int kOccupancy = OCC;                       // waves per SIMD
  static constexpr int kWaves = WM * WN, kNT = 64 * kWaves;
  static constexpr int HM = WM * FM * 16, HN = WN * FN * 16;   // rows of a half
  static constexpr int BM = 2 * HM, BN = 2 * HN;
  static constexpr int kLoads = HM / 8 / kWaves;               // loads of a half per wave
  static_assert(HM == HN, "both operands' halves take as many loads");
};

__device__ __forceinline__ void pin() { __builtin_amdgcn_sched_barrier(0); }

__device__ __forceinline__ void wg_barrier() {
  pin();
  __builtin_amdgcn_s_barrier();
  pin();
}

// The oldest loads but N have arrived.
template <int N>
__device__ __forceinline__ void wait_loads() {
  pin();
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
  pin();
}

__device__ __forceinline__ void wait_lds_reads() {
  pin();
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  pin();
}

// c += a . b with c held in the accumulation registers (ACC; else in the
// others).  Written out, because
// the 256 x 256 tile's accumulators fill all 256 of them and the compiler
// otherwise moves some of them at every step.  The compiler does not see a
// matrix instruction here: what reads c next waits for mfma_done().
template <int WD, bool ACC = true>
__device__ __forceinline__ void mfma_into(f32x4& c, u32x4 a, u32x4 b) {
  if constexpr (WD == BF16 && ACC)
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  else if constexpr (WD == BF16)
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
  else if constexpr (ACC)
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  else
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
}

// The same for 4-bit values, byte SEL of sa and sb the lane's scales.
#define SGMV_MFMA_FP4(C, LO, HI)                                                              \
  asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[" LO "," LO  \
               ",0] op_sel_hi:[" HI "," HI ",0] cbsz:4 blgp:4"                                \
               : "+" C(c) : "v"(a), "v"(b), "v"(sa), "v"(sb))
template <int SEL, bool ACC>
__device__ __forceinline__ void mfma_fp4_into(f32x4& c, u32x4 a, u32x4 b, uint32_t sa, uint32_t sb) {
  if constexpr (ACC) {
    if constexpr (SEL == 0) SGMV_MFMA_FP4("a", "0", "0");
    else if constexpr (SEL == 1) SGMV_MFMA_FP4("a", "1", "0");
    else if constexpr (SEL == 2) SGMV_MFMA_FP4("a", "0", "1");
    else SGMV_MFMA_FP4("a", "1", "1");
  } else {
    if constexpr (SEL == 0) SGMV_MFMA_FP4("v", "0", "0");
    else if constexpr (SEL == 1) SGMV_MFMA_FP4("v", "1", "0");
    else if constexpr (SEL == 2) SGMV_MFMA_FP4("v", "0", "1");
    else SGMV_MFMA_FP4("v", "1", "1");
  }
}
#undef SGMV_MFMA_FP4

// f(0), f(1), ... f(N - 1), the numbers as constants (a loop of this many matrix
// instructions with their scales passes the compiler's limit on unrolling).
template <typename F, int... I>
__device__ __forceinline__ void for_each_of(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void for_each(F f) {
  for_each_of(f, std::make_integer_sequence<int, N>{});
}

// Four words (groups) of four scale bytes (blocks) with rows and columns
// exchanged: word q has the scales of block q of each group.
__device__ __forceinline__ u32x4 transpose_bytes(u32x4 v) {
  const uint32_t a = __builtin_amdgcn_perm(v[1], v[0], 0x05010400);  // v0.0 v1.0 v0.1 v1.1
  const uint32_t b = __builtin_amdgcn_perm(v[3], v[2], 0x05010400);
  const uint32_t c = __builtin_amdgcn_perm(v[1], v[0], 0x07030602);  // v0.2 v1.2 v0.3 v1.3
  const uint32_t d = __builtin_amdgcn_perm(v[3], v[2], 0x07030602);
  return u32x4{__builtin_amdgcn_perm(b, a, 0x05040100), __builtin_amdgcn_perm(b, a, 0x07060302),
               __builtin_amdgcn_perm(d, c, 0x05040100), __builtin_amdgcn_perm(d, c, 0x07060302)};
}

// The larger of a lane's value and the one that DPP control CTRL (of all lanes'
// exchange) brings it.
template <int CTRL>
__device__ __forceinline__ uint32_t lane_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
  return o > v ? o : v;
}

// Operands that other instructions wrote are there for mfma_into.
__device__ __forceinline__ void mfma_ready() {
  pin();
  asm volatile("s_nop 7" ::: "memory");
  pin();
}

// Block `quarter` + 4 s of row `row` of the block-th 16 rows of a half.
__device__ __forceinline__ u32x4 operand_of(const uint16_t* src, int block, int s, int row,
                                            int quarter) {
  return *reinterpret_cast<const u32x4*>(src + (block * 16 + row) * 64 +
                                         ((quarter + 4 * s) ^ (row & 7)) * 8);
}

// More wait states than a matrix instruction takes to write its result.
__device__ __forceinline__ void mfma_done() {
  pin();
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
  pin();
}

template <int WD, int MODE, typename S, bool MX = false>
__global__ __launch_bounds__(S::kNT, S::kOccupancy) void matmul_tiled(MatmulParams p) {
  constexpr int FM = S::FM, FN = S::FN, LL = S::kLoads, HM = S::HM, HN = S::HN;
  constexpr int kS = MX ? (S::BM + S::BN) / S::kNT : 0;  // rows of scales a thread stages
  // Two workgroups a compute unit leave 128 registers of either kind: with the
  // scales more than that are wanted beside the accumulators, and the compiler
  // would move operands between the two right ahead of their use.
  constexpr bool kAcc = !MX || S::kOccupancy == 1;
  __shared__ uint16_t a00[HM * 64], a01[HM * 64], a10[HM * 64], a11[HM * 64];
  // b01 goes on with the staged scales (input rows, then weight rows; 16 bytes each): the
  // compiler makes reads of LDS wait for the loads into the same array that are
  // on their way, or for all loads if there are none, and when scales are read
  // those of b01 have long arrived.
  constexpr int kScales = MX ? (S::BM + S::BN) * 8 : 0;
  __shared__ uint16_t b00[HN * 64], b01[HN * 64 + kScales], b10[HN * 64], b11[HN * 64];
  __shared__ int32_t sh[S::kWaves + 4];

  const TileLoc loc = find_tile<S::kNT>(p, S::BM, sh);
  if (loc.row < 0) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  constexpr int kCols = MODE == kGated ? HN : S::BN;  // output columns of the tile
  const int n0 = loc.col * kCols;
  const int rows = loc.end - loc.row;

  // Input rows: one resource over the tile's rows (or all inputs, gathered),
  // an offset per lane and load.  Weight rows: one resource per half.
  const int lr = lane >> 3;                  // row of a load's eight
  const int chunk = (lane & 7) ^ lr;         // 16-byte block this lane fetches
  const bool gather = (MODE == kGrouped || MODE == kGated) && p.rows != nullptr;
  const rsrc_t xr =
      uniform_rsrc(static_cast<const char*>(p.x) + (gather ? 0 : loc.row) * p.x_row_bytes,
                   ((gather ? p.X : rows) - 1) * p.x_row_bytes + (int64_t)p.H * 2);
  uint32_t xoff[2][LL], woff[LL];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < LL; ++i) {
      const int r = h * HM + (wave * LL + i) * 8 + lr;
      int64_t src = r;
      bool ok = r < rows || (MX && (MODE == kDense || MODE == kAdapted));
      if (gather) {
        src = ok ? p.rows[loc.row + r] : 0;
        ok = ok && src >= 0 && src < p.X;
      }
      xoff[h][i] = ok ? (uint32_t)(src * p.x_row_bytes) + chunk * 16 : kOut;
    }
  rsrc_t wr[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t first = MODE == kGated ? (int64_t)h * p.N + n0 : (int64_t)n0 + h * HN;
    const int64_t left = MODE == kGated ? p.N - n0 : (int64_t)p.N - n0 - h * HN;
    const int64_t nr = left < HN ? left : HN;
    wr[h] = uniform_rsrc(static_cast<const char*>(p.w) + loc.e * p.w_mat_bytes +
                             first * p.w_row_bytes,
                         nr <= 0 ? 0 : (nr - 1) * p.w_row_bytes + (int64_t)p.H * 2);
  }
  // LDS row f 16 + r of a block of 16 FN rows holds the weight row whose
  // products land, over the FN blocks, in one lane's consecutive columns:
  // column (r / 4) 4 FN + 4 f + r % 4.
#pragma unroll
  for (int i = 0; i < LL; ++i) {
    const int q = (wave * LL + i) * 8 + lr;
    const int blk = q / (16 * FN), f = q % (16 * FN) / 16, r = q % 16;
    const int n = blk * 16 * FN + (r >> 2) * 4 * FN + f * 4 + (r & 3);
    woff[i] = (uint32_t)((int64_t)n * p.w_row_bytes) + chunk * 16;
  }

  // MX: this thread's rows of scales, as staged.
  rsrc_t sr[MX ? kS : 1];
  uint32_t soff[MX ? kS : 1];
  if constexpr (MX) {
#pragma unroll
    for (int j = 0; j < kS; ++j) {
      const int u = threadIdx.x + j * S::kNT;
      if (uniform(u) < S::BM) {
        int64_t src = u;
        bool ok = u < rows;
        if (gather) {
          src = ok ? p.rows[loc.row + u] : 0;
          ok = ok && src >= 0 && src < p.X;
        }
        sr[j] = uniform_rsrc(static_cast<const char*>(p.xs) + (gather ? 0 : loc.row) * p.xs_row_bytes,
                             ((gather ? p.X : rows) - 1) * p.xs_row_bytes + p.H / 8);
        soff[j] = ok ? (uint32_t)(src * p.xs_row_bytes) : kOut;
      } else {
        const int q = u - S::BM, h = uniform(q) / HN, in = q % HN, blk = in / (16 * FN);
        const int f = in % (16 * FN) / 16, r = in % 16;
        const int n = blk * 16 * FN + (r >> 2) * 4 * FN + f * 4 + (r & 3);
        const int64_t first = MODE == kGated ? (int64_t)h * p.N + n0 : (int64_t)n0 + h * HN;
        const int64_t left = MODE == kGated ? p.N - n0 : (int64_t)p.N - n0 - h * HN;
        const int64_t nr = left < HN ? left : HN;
        constexpr int kMats = MODE == kGated ? 2 : 1;
        sr[j] = uniform_rsrc(static_cast<const char*>(p.ws) +
                                 limits::stack_row(loc.e, kMats * (int64_t)p.N, first) * p.ws_row_bytes,
                             nr <= 0 ? 0 : (nr - 1) * p.ws_row_bytes + p.H / 8);
        soff[j] = (uint32_t)((int64_t)n * p.ws_row_bytes);
      }
    }
  }

  const int steps = (p.H + 63) / 64;
  // Load i of half h of step t, zeros past the contraction.  The step is part
  // of the lane's offset, which alone is certain to be held against the
  // resource's end (a half of the weights may have no row at all).
  // MX: a load's rows lie a wave-uniform distance from those of the lane's
  // first, whose offset alone takes a register (rows that follow each other
  // and pass the tile's end pass the resource's); the sum is made anew each
  // time, or the compiler keeps all of them.
  auto here = [](int64_t v) __attribute__((always_inline)) {
    uint32_t bytes = (uint32_t)v;
    asm volatile("" : "+s"(bytes));
    return bytes;
  };
  auto load_a = [&](uint16_t* dst, int h, int t, int i) __attribute__((always_inline)) {
    const bool in = t * 64 + 64 <= p.H || t * 64 + chunk * 8 < p.H;
    const uint32_t row = MX && (MODE == kDense || MODE == kAdapted)
                             ? xoff[0][0] + here((h * HM + i * 8) * p.x_row_bytes)
                             : xoff[h][i];
    __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (lds_void*)(dst + (wave * LL + i) * 512), 16,
                                             (int)(in ? row + (uint32_t)t * 128u : kOut), 0,
                                             0, 0);
  };
  auto load_b = [&](uint16_t* dst, int h, int t, int i) __attribute__((always_inline)) {
    const bool in = t * 64 + 64 <= p.H || t * 64 + chunk * 8 < p.H;
    static_assert(16 * FN % (8 * LL) == 0, "a wave's loads of a half stay within a block of rows");
    const uint32_t row =
        MX ? woff[0] + here((i / 2 * 4 + i % 2 * 8 * FN) * p.w_row_bytes) : woff[i];
    __builtin_amdgcn_raw_ptr_buffer_load_lds(wr[h], (lds_void*)(dst + (wave * LL + i) * 512), 16,
                                             (int)(in ? row + (uint32_t)t * 128u : kOut), 0, 0,
                                             0);
  };

  // Operands of part s: row lane & 15 of a block of 16, block lane / 16 + 4 s
  // of the row.
  const int orow = lane & 15, oq = lane >> 4;
  u32x4 xa[3][2 * FM], wb[3][2 * FN];   // three sets of a part's operands
  f32x4 acc[2][2][FM][FN] = {};         // [A half][B half]
  // MX: the lane's offsets within a block, of both parts and in the scales;
  // asm statements in each step keep the compiler from holding their sums with
  // each array's address (34 registers).
  int off[3] = {orow * 64 + (oq ^ (orow & 7)) * 8, orow * 64 + ((oq + 4) ^ (orow & 7)) * 8, orow * 8 + oq * 2};
  auto operand = [&](const uint16_t* src, int block, int s) __attribute__((always_inline)) {
    if constexpr (MX) return *reinterpret_cast<const u32x4*>(src + block * 1024 + off[s]);
    else return operand_of(src, block, s, orow, oq);
  };
  // Operand i of part s into set `to`: the 2 FN of B, then the 2 FM of A.
  auto read_one = [&](const uint16_t* A0, const uint16_t* A1, const uint16_t* B0,
                      const uint16_t* B1, int s, int to, int i) __attribute__((always_inline)) {
    if (i < 2 * FN) wb[to][i] = operand(i < FN ? B0 : B1, wn * FN + i % FN, s);
    else xa[to][i - 2 * FN] = operand(i - 2 * FN < FM ? A0 : A1, wm * FM + (i - 2 * FN) % FM, s);
  };
  // Load i of a step: LL of each half.
  auto load_one = [&](uint16_t* A0, uint16_t* A1, uint16_t* B0, uint16_t* B1, int t,
                      int i) __attribute__((always_inline)) {
    if (i < LL) load_b(B0, 0, t, i);
    else if (i < 2 * LL) load_a(A0, 0, t, i - LL);
    else if (i < 3 * LL) load_b(B1, 1, t, i - 2 * LL);
    else load_a(A1, 1, t, i - 3 * LL);
  };
  constexpr int kReads = 2 * (FM + FN), kLoads = 4 * LL;
  // Loads of a step that part 0 issues, of 16 in large tiles and of 8 in small
  // ones.  10, 12 and all of 16 take 2697, 2695 and 2814 us at 16384 x 28672 x
  // 4096, 3002, 3014 and 3110 us with 64 adapters of rank 64 beside it, 742, 747
  // and 755 us at 8192 x 8192 x 8192.  6 and all of 8 take 45 and 42 us at 512 x
  // 4096 x 4096, 58 and 55 us with adapters; for experts it goes both ways (64 of
  // 96 rows, hidden 2048, 2 x 1408 columns 168 and 159 us; 8 of 102, hidden 2488, 2
  // x 8040 columns 215 and 219; 14 of one, hidden 1040, 2744 columns 19.7 and 20.4).
  constexpr int kEarly = S::kOccupancy == 1                    ? kLoads * 5 / 8
                         : MODE == kDense || MODE == kAdapted ? kLoads
                                                              : kLoads * 3 / 4;
  // MX: scales come for two steps (four groups) at a time.  They are loaded at
  // the start of part 0 of the step before theirs, where a set of operand
  // registers is free, and go to LDS at its end (a line of them serves eight
  // times, so that most come from the L2),
  // a row's four words transposed, so that a lane reads its four groups'
  // scales as one word, and from there into the registers of those they
  // follow, each after its last use.  Words past the row's end, which may be
  // another row's, become zeros.
  u32x4 sraw[MX ? kS : 1];
  uint32_t sa[MX ? 2 * FM : 1], sb[MX ? 2 * FN : 1];
  auto load_scales = [&](int t) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kS; ++j)
      sraw[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                              sr[j], (int)(soff[j] + (uint32_t)t * 8u), 0, 0));
  };
  auto store_scales = [&](int t) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kS; ++j) {
#pragma unroll
      for (int w = 0; w < 4; ++w) sraw[j][w] &= 32 * (2 * t + w) < p.H ? ~0u : 0u;
      *reinterpret_cast<u32x4*>(b01 + HN * 64 + (threadIdx.x + j * S::kNT) * 8) = transpose_bytes(sraw[j]);
    }
  };
  auto read_sa = [&](int m) __attribute__((always_inline)) {
    const int r = (m / FM) * HM + (wm * FM + m % FM) * 16;
    sa[m] = *reinterpret_cast<const uint32_t*>(b01 + HN * 64 + r * 8 + off[2]);
  };
  auto read_sb = [&](int n) __attribute__((always_inline)) {
    const int r = S::BM + (n / FN) * HN + (wn * FN + n % FN) * 16;
    sb[n] = *reinterpret_cast<const uint32_t*>(b01 + HN * 64 + r * 8 + off[2]);
  };
  // Step t, whose operands are in sets 0 and 1 + t % 2, with its LDS
  // (A0, A1, B0, B1) free and the next step's in (C0, C1, D0, D1).  BOTH:
  // whether the second A half holds any row.
  auto step = [&](uint16_t* A0, uint16_t* A1, uint16_t* B0, uint16_t* B1, uint16_t* C0,
                  uint16_t* C1, uint16_t* D0, uint16_t* D1, int t, auto set,
                  auto both) __attribute__((always_inline)) {
    constexpr int kRows = decltype(both)::value ? 2 * FM : FM;
    constexpr int kMfma = kRows * 2 * FN, kSet = decltype(set)::value;
    auto rows_of = [&](auto part, int from, auto between) __attribute__((always_inline)) {
      if constexpr (MX) {
        constexpr int kSel = 2 * (kSet - 1) + decltype(part)::value;
        for_each<kMfma>([&](auto at) __attribute__((always_inline)) {
          constexpr int k = decltype(at)::value, m = k / (2 * FN), n = k % (2 * FN);
          between(k);
          mfma_fp4_into<kSel, kAcc>(acc[m / FM][n / FN][m % FM][n % FN], wb[from][n], xa[from][m], sb[n],
                              sa[m]);
          if constexpr (kSel == 3) {  // the last use of these scales
            pin();
            if constexpr (n == 2 * FN - 1) read_sa(m);
            if constexpr (m == kRows - 1) read_sb(n);
            pin();
          }
        });
      } else {
#pragma unroll
        for (int k = 0; k < kMfma; ++k) {
          const int m = k / (2 * FN), n = k % (2 * FN);
          between(k);
          mfma_into<WD, kAcc>(acc[m / FM][n / FN][m % FM][n % FN], wb[from][n], xa[from][m]);
        }
      }
    };
    int loads = 0, reads = 0;
    if constexpr (MX && kSet == 2) {
      load_scales(t + 1);
      pin();
    }
    rows_of(std::integral_constant<int, 0>{}, 0, [&](int k) __attribute__((always_inline)) {
      if (loads * kMfma <= k * kEarly && loads < kEarly) {
        pin();
        load_one(A0, A1, B0, B1, t + 2, loads++);
        pin();
      }
    });
    wait_loads<kEarly>();
    if constexpr (MX && kSet == 2) {
      store_scales(t + 1);
      wait_lds_reads();
    }
    wg_barrier();
    if constexpr (MX) asm volatile("" : "+v"(off[0]), "+v"(off[1]), "+v"(off[2]));
    rows_of(std::integral_constant<int, 1>{}, kSet, [&](int k) __attribute__((always_inline)) {
      if ((loads - kEarly) * kMfma <= k * (kLoads - kEarly) && loads < kLoads) {
        pin();
        load_one(A0, A1, B0, B1, t + 2, loads++);
        pin();
      }
      // two reads at a time, all of them in three quarters of the part
      if (reads * kMfma * 3 <= k * 8 * kReads && reads < 2 * kReads) {
        pin();
        read_one(C0, C1, D0, D1, reads / kReads, reads < kReads ? 0 : 3 - kSet, reads % kReads);
        ++reads;
        read_one(C0, C1, D0, D1, reads / kReads, reads < kReads ? 0 : 3 - kSet, reads % kReads);
        ++reads;
        pin();
      }
    });
    wait_lds_reads();
    wg_barrier();
  };

  Segment seg{};
  if constexpr (MODE == kAdapted) {
    seg = read_segment(p, threadIdx.x);
    pin();  // ahead of the loads into LDS: loads arrive in order
  }
  if constexpr (MX) {
    load_scales(0);
    pin();  // ahead of the loads into LDS too
  }
#pragma unroll
  for (int i = 0; i < kLoads; ++i) load_one(a00, a01, b00, b01, 0, i);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) load_one(a10, a11, b10, b11, 1, i);
  // Which adapters the tile's rows have, while the first loads are on their way.
  __shared__ int32_t row_pos[MODE == kAdapted ? S::BM : 1], list[MODE == kAdapted ? S::BM : 1];
  __shared__ int32_t segs[MODE == kAdapted ? adapter_words<S::BM>() : 1], count[2], odd_found;
  // float16: exponent 2 e of the values of a row that are staged (and of its
  // accumulators), bit 0 set once e was below zero; and e less the one before.
  constexpr bool kScaled = MODE == kAdapted && WD == F16;
  __shared__ int32_t row_exp[kScaled ? S::BM : 1], row_step[kScaled ? S::BM : 1], any_scaled;
  if constexpr (MODE == kAdapted) {
    // Cleared ahead of tile_adapters' barriers: a tile whose columns no slice
    // covers meets no other one before the flag is read.
    if (threadIdx.x == 0) odd_found = 0;
    if (kScaled && threadIdx.x < S::BM) row_exp[threadIdx.x] = row_step[threadIdx.x] = 0;
    if (kScaled && threadIdx.x == 0) any_scaled = 0;
    tile_adapters<S::kNT, S::BM, false>(p, seg, loc.row, loc.end, row_pos, list, count, segs);
  }
  wait_loads<kLoads>();
  if constexpr (MX) {
    store_scales(0);
    wait_lds_reads();
  }
  wg_barrier();
  if constexpr (MX) {
#pragma unroll
    for (int m = 0; m < 2 * FM; ++m) read_sa(m);
#pragma unroll
    for (int n = 0; n < 2 * FN; ++n) read_sb(n);
  }
#pragma unroll
  for (int i = 0; i < 2 * kReads; ++i)
    read_one(a00, a01, b00, b01, i / kReads, i / kReads, i % kReads);
  wait_lds_reads();
  wg_barrier();
  auto contract = [&](auto both) __attribute__((always_inline)) {
    // Two steps at a time, one of zeros after an odd number: a last single step
    // makes the compiler move accumulators.
    for (int t = 0; t < steps; t += 2) {
      step(a00, a01, b00, b01, a10, a11, b10, b11, t, std::integral_constant<int, 1>{}, both);
      step(a10, a11, b10, b11, a00, a01, b00, b01, t + 1, std::integral_constant<int, 2>{}, both);
    }
  };
  if (rows > HM) contract(std::true_type{});
  else contract(std::false_type{});
  wait_loads<0>();  // the loads past the last step write zeros: none may be on its way at the end
  wait_lds_reads();

  // The thread's number again, so that nothing derived from it below is kept
  // in a register (or worse, in scratch memory, whose reloads would wait for
  // the loads into LDS) during the contraction.
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int erow = tid & 15, eq = (tid >> 4) & 3;

  // Columns of this lane: 4 FN consecutive ones in each B half.
  const int col0 = n0 + wn * 16 * FN + eq * 4 * FN;

  // Adapters, as further steps of the contraction: for each slice and 64 of
  // the rank, the tile's projected rows as two 16-bit parts (A0, A1 of the
  // first buffer the high ones, of the second the low ones) and, one adapter
  // after another, its lora_B rows (alternating between the B buffers, the
  // next ones' loads in flight during these products).  Ranks up to 8, 16 and
  // 32 put 8, 4 and 2 adapters side by side into a step of 64, so that a tile
  // of many single-token requests takes fewer of them.  A row takes
  // part with its own adapter and with zeros elsewhere; so that zero times
  // what another request's weights or another slice's rows hold is nothing,
  // what is not finite is staged as zeros here and its products are added at
  // the end, where they belong.
  [[maybe_unused]] bool odd_values = false;
  if constexpr (MODE == kAdapted) {
    const int adapters = uniform(count[0]);
    constexpr int kA = S::BM * 8 / S::kNT, kB = S::BN * 8 / S::kNT;  // blocks per thread
    // Width of an adapter in a step, log2 of 8 elements, and adapters a step.
    const int wide = p.K <= 8 ? 0 : p.K <= 16 ? 1 : p.K <= 32 ? 2 : 3, side = 8 >> wide;
    // bfloat16 with float32 results: a third part, in the place of the second B
    // buffer (one more barrier an adapter).
    const bool exact = WD == BF16 && p.out_dtype == F32;
    int mine[2 * FM];
#pragma unroll
    for (int m = 0; m < 2 * FM; ++m)
      mine[m] = row_pos[(m / FM) * HM + (wm * FM + m % FM) * 16 + erow];
    [[maybe_unused]] bool scaled = false;  // some row had an exponent but 0
    // The accumulators of row r times 2^step(r), where any of the wave's rows
    // takes another exponent.
    auto rescale = [&](auto step) __attribute__((always_inline)) {
      int by[2 * FM];
      bool any = false;
#pragma unroll
      for (int m = 0; m < 2 * FM; ++m) {
        by[m] = step((m / FM) * HM + (wm * FM + m % FM) * 16 + erow);
        any = any || by[m] != 0;
      }
      if (__ballot(any) == 0) return;
      mfma_done();
#pragma unroll
      for (int m = 0; m < 2 * FM; ++m)
#pragma unroll
        for (int n = 0; n < 2 * FN; ++n) {
          // The copy is made here and goes back before the next one's: the
          // compiler would hold all of them in vector registers otherwise.
          f32x4& c = acc[m / FM][n / FN][m % FM][n % FN];
          if constexpr (kAcc) asm volatile("" : "+a"(c));
#pragma unroll
          for (int j = 0; j < 4; ++j) c[j] = ldexpf(c[j], by[m]);
          if constexpr (kAcc) asm volatile("" : "+a"(c));
          pin();
        }
      mfma_ready();
    };
    for (int sl = 0; sl < (adapters > 0 ? p.num_slices : 0); ++sl) {
      const AdapterDesc d = adapter_desc(sl);
      if (d.offset >= n0 + S::BN || d.offset + d.n <= n0) continue;
      const rsrc_t vr = uniform_rsrc(
          reinterpret_cast<const char*>(d.v + (int64_t)loc.row * p.v_stride),
          (int64_t)rows * p.v_stride * 4);
      for (int k = 0; k < p.K; k += 64) {
        u32x4 nb[kB];
        auto load_lora_b = [&](int i) __attribute__((always_inline)) {
#pragma unroll
          for (int j = 0; j < kB; ++j) {
            const int u = tid + j * S::kNT, q = u >> 3, c = u & 7;
            const int h = q / HN, in = q % HN, blk = in / (16 * FN);
            const int f = in % (16 * FN) / 16, r = in % 16;
            const int n = n0 + h * HN + blk * 16 * FN + (r >> 2) * 4 * FN + f * 4 + (r & 3) -
                          (int)d.offset;
            const int pos = i + (c >> wide), at = k + ((c & ((1 << wide) - 1)) << 3);
            const bool ok = n >= 0 && n < d.n && pos < adapters && at < p.K;
            const int64_t e = ok ? ((int64_t)list[ok ? pos : 0] * d.n + n) * p.K + at : 0;
            load_vec8<WD>(d.b, e, &nb[j]);  // the stack's first block where there is none
#pragma unroll
            for (int w = 0; w < 4; ++w) nb[j][w] = ok ? nb[j][w] : 0u;
          }
        };
        auto store_lora_b = [&](uint16_t* B0, uint16_t* B1) __attribute__((always_inline)) {
          bool found = false;
#pragma unroll
          for (int j = 0; j < kB; ++j) {
            const int u = tid + j * S::kNT, q = u >> 3, c = u & 7;
            uint16_t* dst = q < HN ? B0 : B1;
            u32x4 v = nb[j];
            if (any_odd<WD>(v)) {
              v = drop_odd<WD>(v);
              found = true;
            }
            *reinterpret_cast<u32x4*>(dst + (q % HN) * 64 + ((c ^ (q & 7)) * 8)) = v;
          }
          if (found) odd_found = 1;
        };
        load_lora_b(0);
        __syncthreads();  // the LDS is free: last step's or last round's reads are over
        float v[kA][8];  // all loads ahead of the branches below: they arrive together
        uint32_t most[kA], worst = 0;
#pragma unroll
        for (int j = 0; j < kA; ++j) {
          const int u = tid + j * S::kNT, r = u >> 3, c = u & 7;
          u32x4 raw[2];
          const int at = k + ((c & ((1 << wide) - 1)) << 3);
          buf_load8<F32>(vr, at < p.K ? (uint32_t)(r * p.v_stride + at) * 4u : kOut, raw);
          out_values<F32>(raw, v[j]);
        }
#pragma unroll
        for (int j = 0; j < kA; ++j) {
          most[j] = largest_of(v[j]);
          worst = most[j] > worst ? most[j] : worst;
        }
        if (worst >= kOddBits) {
#pragma unroll
          for (int j = 0; j < kA; ++j) {
            // a row of no segment may hold anything
            if (most[j] >= kOddBits && row_pos[(tid + j * S::kNT) >> 3] >= 0) odd_found = 1;
            drop_odd(v[j]);
            most[j] = largest_of(v[j]);
          }
        }
        if constexpr (kScaled) {
          int e[kA];
          bool some = scaled;
#pragma unroll
          for (int j = 0; j < kA; ++j) {  // eight lanes have the row's values
            most[j] = lane_max<0xB1>(most[j]);
            most[j] = lane_max<0x4E>(most[j]);
            most[j] = lane_max<0x141>(most[j]);
            e[j] = split_exponent(most[j]);
            some = some || e[j] != 0;
          }
          if (some) {
#pragma unroll
            for (int j = 0; j < kA; ++j) {
              const int u = tid + j * S::kNT, r = u >> 3;
              // Rows whose values were large once stay at the exponent that
              // these took or 0: their accumulators times 2^40 might overflow.
              const int32_t was = row_exp[r];
              if (row_pos[r] < 0 || ((was & 1) && e[j] > 0)) e[j] = 0;
              scale_values(v[j], e[j]);
              if ((u & 7) == 0) {
                row_step[r] = e[j] - (was >> 1);
                row_exp[r] = 2 * e[j] | (was & 1) | (e[j] < 0);
                if (e[j] != 0) any_scaled = 1;
              }
            }
          }
        }
#pragma unroll
        for (int j = 0; j < kA; ++j) {
          const int u = tid + j * S::kNT, r = u >> 3, c = u & 7;
          u32x4 hi, lo;
          split_operand<WD>(v[j], &hi, &lo);
          const int to = (r % HM) * 64 + ((c ^ (r & 7)) * 8);
          if (exact) *reinterpret_cast<u32x4*>((r < HM ? b10 : b11) + to) = third_operand(v[j]);
          *reinterpret_cast<u32x4*>((r < HM ? a00 : a01) + to) = hi;
          *reinterpret_cast<u32x4*>((r < HM ? a10 : a11) + to) = lo;
        }
        store_lora_b(b00, b01);
        __syncthreads();
        if constexpr (kScaled) {
          scaled = uniform(any_scaled) != 0;
          if (scaled) rescale([&](int r) { return row_step[r]; });
        }
        bool odd = false;
        for (int i = 0; i < adapters; i += side, odd = !odd && !exact) {
          if (i + side < adapters) load_lora_b(i + side);
          const uint16_t* B0 = odd ? b10 : b00;
          const uint16_t* B1 = odd ? b11 : b01;
          // the second 32 hold something: more of the rank, or more adapters
          const int subs = (side == 1 ? p.K - k > 32 : i + side / 2 < adapters) ? 2 : 1;
          for (int s = 0; s < subs; ++s) {
            const int slot = i + ((eq + 4 * s) >> wide);  // the adapter of this lane's block
#pragma unroll
            for (int n = 0; n < 2 * FN; ++n) wb[0][n] = operand_of(n < FN ? B0 : B1, wn * FN + n % FN, s, erow, eq);
#pragma unroll
            for (int m = 0; m < 2 * FM; ++m) {
              if (__ballot(mine[m] == slot) == 0) continue;  // none of these 16 rows
#pragma unroll
              for (int part = 2; part >= 0; --part) {
                if (part == 2 && !exact) continue;
                const uint16_t* A = m < FM ? (part == 0 ? a00 : part == 1 ? a10 : b10)
                                           : (part == 0 ? a01 : part == 1 ? a11 : b11);
                u32x4 x = operand_of(A, wm * FM + m % FM, s, erow, eq);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = mine[m] == slot ? x[j] : 0u;
                mfma_ready();
#pragma unroll
                for (int n = 0; n < 2 * FN; ++n)
                  mfma_into<WD, kAcc>(acc[m / FM][n / FN][m % FM][n % FN], wb[0][n], x);
              }
            }
          }
          if (i + side < adapters) {
            if (exact) __syncthreads();  // every wave has read the weights there
            if (odd || exact) store_lora_b(b00, b01);
            else store_lora_b(b10, b11);
          }
          __syncthreads();
        }
      }
    }
    if (scaled) rescale([&](int r) { return -(row_exp[r] >> 1); });
    odd_values = adapters > 0 && uniform(odd_found) != 0;
    if (odd_values) {  // the A buffers, free now, take a code for every result
#pragma unroll 1
      for (int u = tid; u < S::BM * S::BN; u += S::kNT) {
        const int r = u / S::BN, c = u % S::BN;
        if (r < rows && n0 + c < p.N) {
          uint16_t* part = r < HM ? (r < HM / 2 ? a00 : a01) : (r < HM + HM / 2 ? a10 : a11);
          const float odd =
              odd_products<WD>(p, loc.row + r, row_pos[r] < 0 ? -1 : list[row_pos[r]], n0 + c);
          // 0 nothing, 1 +inf, 2 -inf, 3 NaN
          reinterpret_cast<uint8_t*>(part)[r % (HM / 2) * S::BN + c] =
              odd == 0.f ? 0 : odd != odd ? 3 : odd > 0.f ? 1 : 2;
        }
      }
      __syncthreads();
    }
  }
  mfma_done();

  // Results: eight consecutive columns of a token per lane and access, with
  // rows and columns past the tile's sent past the buffer's end instead of
  // branched around.  VEC: 16-byte accesses, else element by element.
  const rsrc_t orsrc = uniform_rsrc(static_cast<const char*>(p.out) + loc.row * p.out_row_bytes,
                                    (int64_t)rows * p.out_row_bytes);
  const rsrc_t brsrc = uniform_rsrc(static_cast<const char*>(p.bias), (int64_t)p.N * 2);
  auto finish = [&](auto od, auto vec) __attribute__((always_inline)) {
    constexpr int OD = decltype(od)::value;
    constexpr bool VEC = decltype(vec)::value;
    constexpr uint32_t ob = OD == F32 ? 4 : 2;
#pragma unroll
    for (int bh = 0; bh < (MODE == kGated ? 1 : 2); ++bh)
#pragma unroll
      for (int g = 0; g < FN / 2; ++g) {
        const int col = col0 + bh * HN + g * 8;
        float bias[8] = {};
        if constexpr (MODE == kDense || MODE == kAdapted) {
          if (p.bias) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              bias[j] = widen<WD>((uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(
                  brsrc, (int)((uint32_t)(col + j) * 2u), 0, 0));
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int m = 0; m < FM; ++m) {
            const int r = h * HM + (wm * FM + m) * 16 + erow;
            const uint32_t off = (uint32_t)(r * p.out_row_bytes) + (uint32_t)col * ob;
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int f = 2 * g + j / 4;
              y[j] = MODE == kGated ? gate(acc[h][0][m][f][j & 3], acc[h][1][m][f][j & 3])
                                    : acc[h][bh][m][f][j & 3] + bias[j];
            }
            if constexpr (MODE == kAdapted) {
              if (odd_values) {
                const uint16_t* half = h == 0 ? (r < HM / 2 ? a00 : a01)
                                              : (r < HM + HM / 2 ? a10 : a11);
                const uint2 codes = *reinterpret_cast<const uint2*>(
                    reinterpret_cast<const uint8_t*>(half) + r % (HM / 2) * S::BN + col - n0);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const uint32_t c = (j < 4 ? codes.x : codes.y) >> (8 * (j & 3)) & 3u;
                  y[j] += c == 0 ? 0.f : c == 1 ? INFINITY : c == 2 ? -INFINITY : NAN;
                }
              }
            }
            u32x4 raw[raw_vecs<OD>()];
            if constexpr (VEC) {
              const uint32_t at = r < rows && col < p.N ? off : kOut;
              if constexpr (MODE == kDense || MODE == kAdapted) {
                if (p.add) {
                  float o[8];
                  buf_load8<OD>(orsrc, at, raw);
                  out_values<OD>(raw, o);
#pragma unroll
                  for (int j = 0; j < 8; ++j) y[j] += o[j];
                }
              }
              out_pack<OD>(y, raw);
              buf_store8<OD>(orsrc, at, raw);
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const int at = (int)(r < rows && col + j < p.N ? off + j * ob : kOut);
                float o = 0.f;
                if constexpr (OD == F32) {
                  if (p.add)
                    o = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(orsrc, at, 0, 0));
                  __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(y[j] + o), orsrc, at, 0, 0);
                } else {
                  if (p.add)
                    o = widen<OD>((uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(orsrc, at,
                                                                                           0, 0));
                  __builtin_amdgcn_raw_buffer_store_b16((uint16_t)pack2<OD>(y[j] + o, 0.f), orsrc,
                                                        at, 0, 0);
                }
              }
            }
            pin();  // one block's values at a time: the accumulators' copies must not pile up
          }
      }
  };
  auto finish_as = [&](auto vec) __attribute__((always_inline)) {
    if (p.out_dtype == BF16) finish(std::integral_constant<int, BF16>{}, vec);
    else if (p.out_dtype == F16) finish(std::integral_constant<int, F16>{}, vec);
    else finish(std::integral_constant<int, F32>{}, vec);
  };
  if (p.vec_out) finish_as(std::true_type{});
  else finish_as(std::false_type{});
}

}  // namespace dev
}  // namespace sgmv
