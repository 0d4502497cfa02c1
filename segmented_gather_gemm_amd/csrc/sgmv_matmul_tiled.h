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
// A wave owns a quarter of its output in each pair of halves and goes through
// them in four phases per step, (A0, Bx), (A0, By), (A1, By), (A1, Bx), with
// the next step's x this step's y: a phase reads one new half into
// registers, and the operands take 64 registers beside the accumulators'
// 128.  Counting phases and halves in this order, phase q reads half q + 1
// and refills the LDS of half q, which every wave has read, with half q + 8;
// loads have six phases to arrive.  With eight waves the two waves of a SIMD
// run half a phase apart: while one issues its matrix instructions, the other
// reads its next operands and issues loads, and a barrier after each half
// phase keeps them so.
#pragma once

#include <type_traits>

#include "sgmv_matmul.h"

namespace sgmv {
namespace dev {

enum { kDense = 0, kGrouped = 1, kGated = 2 };

typedef __attribute__((address_space(3))) void lds_void;

// The shape of a tiled kernel: WM x WN waves, each FM x FN blocks of 16 x 16
// per pair of halves.
template <int WM_, int WN_, int FM_, int FN_>
struct TileShape {
  static constexpr int WM = WM_, WN = WN_, FM = FM_, FN = FN_;
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

template <int WD, int MODE, typename S>
__global__ __launch_bounds__(S::kNT, 2) void matmul_tiled(MatmulParams p) {
  constexpr int FM = S::FM, FN = S::FN, LL = S::kLoads, HM = S::HM, HN = S::HN;
  constexpr bool kOffset = S::kWaves == 8;
  __shared__ uint16_t a00[HM * 64], a01[HM * 64], a10[HM * 64], a11[HM * 64];
  __shared__ uint16_t b00[HN * 64], b01[HN * 64], b10[HN * 64], b11[HN * 64];
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
  const bool gather = MODE != kDense && p.rows != nullptr;
  const rsrc_t xr =
      make_rsrc(static_cast<const char*>(p.x) + (gather ? 0 : loc.row) * p.x_row_bytes,
                ((gather ? p.X : rows) - 1) * p.x_row_bytes + (int64_t)p.H * 2);
  uint32_t xoff[2][LL], woff[LL];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < LL; ++i) {
      const int r = h * HM + (wave * LL + i) * 8 + lr;
      int64_t src = r;
      bool ok = r < rows;
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
    wr[h] = make_rsrc(static_cast<const char*>(p.w) + loc.e * p.w_mat_bytes + first * p.w_row_bytes,
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

  // Loads of half h of step t (nothing past the contraction).
  auto load_a = [&](uint16_t* dst, int h, int t) __attribute__((always_inline)) {
    const bool in = t * 64 + chunk * 8 < p.H;
#pragma unroll
    for (int i = 0; i < LL; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          xr, (lds_void*)(dst + (wave * LL + i) * 512), 16,
          (int)(in ? xoff[h][i] + (uint32_t)t * 128u : kOut), 0, 0, 0);
  };
  auto load_b = [&](uint16_t* dst, int h, int t) __attribute__((always_inline)) {
    const bool in = t * 64 + chunk * 8 < p.H;
#pragma unroll
    for (int i = 0; i < LL; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          wr[h], (lds_void*)(dst + (wave * LL + i) * 512), 16,
          (int)(in ? woff[i] + (uint32_t)t * 128u : kOut), 0, 0, 0);
  };

  // Operands: row lane & 15 of a block of 16, block lane / 16 + 4 s of the
  // row.  A wave whose rows of a half all lie past the tile skips them.
  const int orow = lane & 15, oq = lane >> 4;
  const bool live[2] = {wm * FM * 16 < rows, HM + wm * FM * 16 < rows};
  u32x4 xa[FM][2], wb[2][FN][2];
  f32x4 acc[2][2][FM][FN] = {};   // [A half][B half]
  auto read_a = [&](const uint16_t* src, int h) __attribute__((always_inline)) {
    if (!live[h]) return;
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
      for (int s = 0; s < 2; ++s)
        xa[f][s] = *reinterpret_cast<const u32x4*>(src + ((wm * FM + f) * 16 + orow) * 64 +
                                                   ((oq + 4 * s) ^ (orow & 7)) * 8);
  };
  auto read_b = [&](const uint16_t* src, int h) __attribute__((always_inline)) {
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
      for (int s = 0; s < 2; ++s)
        wb[h][f][s] = *reinterpret_cast<const u32x4*>(src + ((wn * FN + f) * 16 + orow) * 64 +
                                                      ((oq + 4 * s) ^ (orow & 7)) * 8);
  };
  // The second half of a phase, between barriers.
  auto products = [&](int ah, int bh) __attribute__((always_inline)) {
    wait_loads<6 * LL>();
    wait_lds_reads();
    wg_barrier();
    if (live[ah]) {
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int m = 0; m < FM; ++m)
#pragma unroll
          for (int n = 0; n < FN; ++n)
            acc[ah][bh][m][n] = mfma<WD>(wb[bh][n][s], xa[m][s], acc[ah][bh][m][n]);
      __builtin_amdgcn_s_setprio(0);
    }
    wg_barrier();
  };
  // One step: its halves' LDS, the next step's first B half, x and y.
  auto step = [&](uint16_t* A0, uint16_t* A1, uint16_t* Bx, uint16_t* By, uint16_t* next, int x,
                  int t) __attribute__((always_inline)) {
    const int y = 1 - x;
    read_a(A0, 0);
    load_b(Bx, x, t + 2);
    products(0, x);
    read_b(By, y);
    load_a(A0, 0, t + 2);
    products(0, y);
    read_a(A1, 1);
    load_b(By, y, t + 2);
    products(1, y);
    read_b(next, y);
    load_a(A1, 1, t + 2);
    products(1, x);
  };

  const int steps = (p.H + 63) / 64;
  load_b(b00, 0, 0);
  load_a(a00, 0, 0);
  load_b(b01, 1, 0);
  load_a(a01, 1, 0);
  load_b(b11, 1, 1);
  load_a(a10, 0, 1);
  load_b(b10, 0, 1);
  load_a(a11, 1, 1);
  wait_loads<6 * LL>();
  wg_barrier();
  read_b(b00, 0);
  if (kOffset && wave >= S::kWaves / 2) wg_barrier();  // half a phase behind
  int t = 0;
  for (; t + 1 < steps; t += 2) {
    step(a00, a01, b00, b01, b11, 0, t);
    step(a10, a11, b11, b10, b00, 1, t + 1);
  }
  if (t < steps) step(a00, a01, b00, b01, b11, 0, t);
  if (kOffset && wave < S::kWaves / 2) wg_barrier();
  wait_loads<0>();  // the loads past the last step write zeros: none may be on its way at the end
  wait_lds_reads();

  // Columns of this lane: 4 FN consecutive ones in each B half.
  const int col0 = n0 + wn * 16 * FN + oq * 4 * FN;

  if constexpr (MODE == kDense) {
    if (p.num_slices > 0) {
      __shared__ int32_t row_a[S::BM] __attribute__((aligned(16)));
      __shared__ int32_t list[S::BM];
      __shared__ int32_t count;
      tile_adapters<S::kNT, S::BM>(p, loc.row, loc.end, row_a, list, &count);
      const int32_t adapters = uniform(count);
      for (int i = 0; i < adapters; ++i) {
        const int32_t a = uniform(list[i]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          bool mine[FM];
          uint64_t any = 0;
#pragma unroll
          for (int m = 0; m < FM; ++m) {
            mine[m] = row_a[h * HM + (wm * FM + m) * 16 + orow] == a;
            any |= __ballot(mine[m]);
          }
          if (any == 0) continue;
          for (int sl = 0; sl < p.num_slices; ++sl) {
            const AdapterDesc& d = p.s[sl];
            if (d.offset >= n0 + S::BN || d.offset + d.n <= n0) continue;
            const bool vb = ((reinterpret_cast<uintptr_t>(d.b) & 15) == 0) && p.K % 8 == 0;
            for (int k = 0; k < p.K; k += 32) {
              const int at = k + oq * 8, cnt = clamp8((int64_t)p.K - at);
              u32x4 hi[FM], lo[FM];
#pragma unroll
              for (int m = 0; m < FM; ++m) {
                const int64_t row = loc.row + h * HM + (wm * FM + m) * 16 + orow;
                u32x4 raw[2];
                load_any8<F32>(d.v, row * p.v_stride + at, mine[m] ? cnt : 0, true, raw);
                float v[8];
                out_values<F32>(raw, v);
                split_operand<WD>(v, &hi[m], &lo[m]);
              }
#pragma unroll
              for (int bh = 0; bh < 2; ++bh)
#pragma unroll
                for (int f = 0; f < FN; ++f) {
                  const int64_t n = (int64_t)n0 + bh * HN + wn * 16 * FN +
                                    (orow >> 2) * 4 * FN + f * 4 + (orow & 3) - d.offset;
                  const bool in = n >= 0 && n < d.n;
                  u32x4 bv;
                  load_any8<WD>(d.b, ((int64_t)a * d.n + (in ? n : 0)) * p.K + at, in ? cnt : 0,
                                vb, &bv);
#pragma unroll
                  for (int m = 0; m < FM; ++m) {
                    acc[h][bh][m][f] = mfma<WD>(bv, hi[m], acc[h][bh][m][f]);
                    acc[h][bh][m][f] = mfma<WD>(bv, lo[m], acc[h][bh][m][f]);
                  }
                }
            }
          }
        }
      }
    }
  }

  auto finish = [&](auto od) __attribute__((always_inline)) {
    constexpr int OD = decltype(od)::value;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        const int r = h * HM + (wm * FM + m) * 16 + orow;
        if (r >= rows) continue;
        char* out = static_cast<char*>(p.out) + (int64_t)(loc.row + r) * p.out_row_bytes;
#pragma unroll
        for (int bh = 0; bh < (MODE == kGated ? 1 : 2); ++bh)
#pragma unroll
          for (int g = 0; g < FN / 2; ++g) {  // eight columns at a time
            const int col = col0 + bh * HN + g * 8;
            const int cnt = clamp8((int64_t)p.N - col);
            if (cnt == 0) continue;
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int f = 2 * g + j / 4;
              y[j] = MODE == kGated ? gate(acc[h][0][m][f][j & 3], acc[h][1][m][f][j & 3])
                                    : acc[h][bh][m][f][j & 3];
            }
            if constexpr (MODE == kDense) {
              if (p.bias) {
                u32x4 raw;
                float b[8];
                load_any8<WD>(p.bias, col, cnt, p.vec_bias, &raw);
                out_values<WD>(&raw, b);
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] += b[j];
              }
              if (p.add) {
                u32x4 raw[raw_vecs<OD>()];
                float o[8];
                load_any8<OD>(out, col, cnt, p.vec_out, raw);
                out_values<OD>(raw, o);
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] += o[j];
              }
            }
            store_any8<OD>(out, col, cnt, p.vec_out, y);
          }
      }
  };
  if (p.out_dtype == BF16) finish(std::integral_constant<int, BF16>{});
  else if (p.out_dtype == F16) finish(std::integral_constant<int, F16>{});
  else finish(std::integral_constant<int, F32>{});
}

}  // namespace dev
}  // namespace sgmv
