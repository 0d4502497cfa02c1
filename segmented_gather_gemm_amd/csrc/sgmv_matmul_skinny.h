// sgmv_matmul_skinny.h -- gfx950 kernel of the shared projection with adapters
// and of the grouped products for few rows (decode batches, single tokens).
// Internal to libsgmv.
//
// A few rows against a whole weight matrix are bound by reading the weights
// once, so the kernel is built to keep loads in flight: a workgroup of eight
// waves computes 16 MB rows x 16 NB columns, the waves take steps of 64 along
// the contraction in turn (wave w steps w, w + 8, ...), and every wave loads
// its weights and input rows straight into matrix-instruction registers, G
// steps ahead of their use.  No wave waits for another until the end, where
// the eight partial sums meet in LDS and are added in order.  Splitting the
// contraction inside the workgroup gives a 4096-wide projection 256
// workgroups of 16 columns, with no partial sums in memory.
//
// Measured (bfloat16, hidden 4096, weights from memory, us a call): one row, 4096
// columns 9.9 (3.4 TB/s; the launch and the first loads' latency are about half
// of it), 14336 columns 25.5 (4.6 TB/s); 17 rows, 4096 columns 12.4; 64 rows with
// 32 adapters through 6144 columns 49.8, 40 of them this kernel's, where the
// operands of 64 rows through one compute unit's L1 bind (768 KiB a
// workgroup).  Two steps ahead, against one and four: 10.0, 10.1 and 9.7 for
// one row, 17.8, 18.6 and 17.5 with its adapter, 15.2, 14.1 and 16.7 for 32 rows,
// 17.0, 16.2 and 17.6 for 4 gated experts of 4 rows (hidden 2048, 2 x 1408).  16
// columns a workgroup against 32: 10.0 and 12.8 for one row, 15.2 and 20.1 for
// 32; 64 rows with 32 adapters take 32 columns, 49.8 and 75.6 (with 4 adapters
// and 4096 columns 44.4 and 39.1).
#pragma once

#include "sgmv_matmul.h"

namespace sgmv {
namespace dev {

constexpr int kSkinnyWaves = 8;

template <int WD, int MODE, int MB, int NB, int G>
__global__ __launch_bounds__(64 * kSkinnyWaves, 2) void matmul_skinny(MatmulParams p) {
  constexpr int kW = kSkinnyWaves, kNT = 64 * kW, ROWS = 16 * MB;
  constexpr int kMats = MODE == kGated ? 2 : 1;   // weight blocks per column block
  constexpr int kBlocks = MB * NB * kMats, kPad = 20;
  __shared__ int32_t sh[kW + 4];
  __shared__ float part[kW][kBlocks][16][kPad];
  const TileLoc loc = find_tile<kNT>(p, ROWS, sh);
  if (loc.row < 0) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int n0 = loc.col * 16 * NB, rows = loc.end - loc.row;
  const int lr = lane & 15, lq = lane >> 4;

  const bool gather = (MODE == kGrouped || MODE == kGated) && p.rows != nullptr;
  const rsrc_t xr =
      uniform_rsrc(static_cast<const char*>(p.x) + (gather ? 0 : loc.row) * p.x_row_bytes,
                   ((gather ? p.X : rows) - 1) * p.x_row_bytes + (int64_t)p.H * 2);
  uint32_t xoff[MB];
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const int r = m * 16 + lr;
    int64_t src = r;
    bool ok = r < rows;
    if (gather) {
      src = ok ? p.rows[loc.row + r] : 0;
      ok = ok && src >= 0 && src < p.X;
    }
    xoff[m] = ok ? (uint32_t)(src * p.x_row_bytes) : kOut;
  }
  rsrc_t wr[kMats];
#pragma unroll
  for (int g = 0; g < kMats; ++g) {
    const int64_t nr = p.N - n0 < 16 * NB ? p.N - n0 : 16 * NB;
    wr[g] = uniform_rsrc(static_cast<const char*>(p.w) + loc.e * p.w_mat_bytes +
                             ((int64_t)g * p.N + n0) * p.w_row_bytes,
                         (nr - 1) * p.w_row_bytes + (int64_t)p.H * 2);
  }
  uint32_t woff[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) woff[n] = (uint32_t)((n * 16 + lr) * p.w_row_bytes);

  // Step u of this wave is step w + 8 u of the contraction: 64 elements, two
  // matrix instructions; lane quarter q holds blocks q and 4 + q of a row.
  const int steps = (p.H + 63) / 64;
  const int mine = (steps - wave + kW - 1) / kW;
  u32x4 wv[G][kMats][NB][2], xv[G][MB][2];
  f32x4 acc[kMats][MB][NB] = {};
  auto load = [&](int g, int u) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int k = (wave + u * kW) * 64 + s * 32 + lq * 8;
      const bool in = u < mine && k < p.H;
#pragma unroll
      for (int t = 0; t < kMats; ++t)
#pragma unroll
        for (int n = 0; n < NB; ++n)
          buf_load8<WD>(wr[t], in ? woff[n] + k * 2u : kOut, &wv[g][t][n][s]);
#pragma unroll
      for (int m = 0; m < MB; ++m) buf_load8<WD>(xr, in ? xoff[m] + k * 2u : kOut, &xv[g][m][s]);
    }
  };
  Segment seg{};
  if constexpr (MODE == kAdapted) seg = read_segment(p, threadIdx.x);
#pragma unroll
  for (int g = 0; g < G; ++g) load(g, g);
  // Which adapters the tile's rows have, while the first loads are on their way.
  __shared__ int32_t row_pos[MODE == kAdapted ? ROWS : 1], list[MODE == kAdapted ? ROWS : 1];
  __shared__ int32_t segs[MODE == kAdapted ? adapter_words<ROWS>() : 1], count[2], odd_found;
  if constexpr (MODE == kAdapted) {
    if (threadIdx.x == 0) odd_found = 0;  // ahead of tile_adapters' barriers
    tile_adapters<kNT, ROWS, true>(p, seg, loc.row, loc.end, row_pos, list, count, segs);
  }
  for (int u = 0; u < mine; u += G) {
#pragma unroll
    for (int g = 0; g < G; ++g) {  // past the last step: zeros
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int t = 0; t < kMats; ++t)
#pragma unroll
          for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int n = 0; n < NB; ++n)
              acc[t][m][n] = mfma<WD>(wv[g][t][n][s], xv[g][m][s], acc[t][m][n]);
      load(g, u + G + g);
    }
  }

  // Adapters, dealt to the waves, kAtOnce of a wave's own at a time: each
  // adapter's products go to the lanes whose token has it, so that what one
  // request's weights hold never reaches another's rows.
  if constexpr (MODE == kAdapted) {
    constexpr int kAtOnce = 4;
    const int adapters = uniform(count[0]);
    int pos[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) pos[m] = row_pos[m * 16 + lr];
    for (int sl = 0; sl < (wave < adapters ? p.num_slices : 0); ++sl) {
      const AdapterDesc ad = adapter_desc(sl);
      if (ad.offset >= n0 + 16 * NB || ad.offset + ad.n <= n0) continue;
      const rsrc_t vr =
          uniform_rsrc(reinterpret_cast<const char*>(ad.v + (int64_t)loc.row * p.v_stride),
                       (int64_t)rows * p.v_stride * 4);
      for (int k = 0; k < p.K; k += 32) {
        const int at = k + lq * 8;
        u32x4 raw[MB][2], hi[MB], lo[MB];
        [[maybe_unused]] u32x4 third[MB];  // bfloat16 with float32 results
        const bool exact = WD == BF16 && p.out_dtype == F32;
        [[maybe_unused]] int e[MB];  // float16: exponent of a token's values in the parts
#pragma unroll
        for (int m = 0; m < MB; ++m)
          buf_load8<F32>(vr, at < p.K ? (uint32_t)((m * 16 + lr) * p.v_stride + at) * 4u : kOut,
                         raw[m]);
        for (int i = wave; i < adapters; i += kW * kAtOnce) {
          u32x4 bv[kAtOnce][NB];
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
            const int a = uniform(list[i + j * kW < adapters ? i + j * kW : i]);
            const rsrc_t br = uniform_rsrc(static_cast<const char*>(ad.b) + a * ad.n * p.K * 2,
                                           ad.n * p.K * 2);
#pragma unroll
            for (int n = 0; n < NB; ++n) {
              const int c = n0 + n * 16 + lr - (int)ad.offset;
              buf_load8<WD>(br,
                            c >= 0 && c < ad.n && at < p.K ? (uint32_t)(c * p.K + at) * 2u : kOut,
                            &bv[j][n]);
            }
          }
          if (i == wave) {
#pragma unroll
            for (int m = 0; m < MB; ++m) {
              float v[8];
              out_values<F32>(raw[m], v);
              if (any_odd(v)) {
                drop_odd(v);
                if (pos[m] >= 0) odd_found = 1;  // else no segment's row: anything may be there
              }
              if constexpr (WD == F16) {  // a token's 32 values are in the lanes lr + 16 q
                e[m] = split_exponent(quarters_max(largest_of(v)));
                scale_values(v, e[m]);
              }
              split_operand<WD>(v, &hi[m], &lo[m]);
              if (exact) third[m] = third_operand(v);
            }
          }
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
            if (i + j * kW >= adapters) continue;
            bool odd = false;
#pragma unroll
            for (int n = 0; n < NB; ++n) odd = odd || any_odd<WD>(bv[j][n]);
            if (__ballot(odd) != 0) {
              odd_found = 1;
#pragma unroll
              for (int n = 0; n < NB; ++n) bv[j][n] = drop_odd<WD>(bv[j][n]);
            }
#pragma unroll
            for (int m = 0; m < MB; ++m) {
              const bool own = pos[m] == i + j * kW;
              if (__ballot(own) == 0) continue;
              f32x4 d[NB] = {};
              if (exact) {
#pragma unroll
                for (int n = 0; n < NB; ++n) d[n] = mfma<WD>(bv[j][n], third[m], d[n]);
              }
#pragma unroll
              for (int n = 0; n < NB; ++n) {
                d[n] = mfma<WD>(bv[j][n], lo[m], d[n]);
                d[n] = mfma<WD>(bv[j][n], hi[m], d[n]);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const float y = WD == F16 ? ldexpf(d[n][q], -e[m]) : d[n][q];
                  acc[0][m][n][q] += own ? y : 0.f;
                }
              }
            }
          }
        }
      }
    }
  }

#pragma unroll
  for (int t = 0; t < kMats; ++t)
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int n = 0; n < NB; ++n)
        *reinterpret_cast<f32x4*>(&part[wave][(t * MB + m) * NB + n][lr][lq * 4]) = acc[t][m][n];
  __syncthreads();
  [[maybe_unused]] bool odd_values = false;
  if constexpr (MODE == kAdapted) odd_values = uniform(odd_found) != 0;
  for (int e = threadIdx.x; e < ROWS * 16 * NB; e += kNT) {
    const int c = e % (16 * NB), r = e / (16 * NB), n = c / 16, m = r / 16;
    const int col = n0 + c;
    if (r >= rows || col >= p.N) continue;
    float y[kMats];
#pragma unroll
    for (int t = 0; t < kMats; ++t) {
      y[t] = 0.f;
#pragma unroll
      for (int w = 0; w < kW; ++w) y[t] += part[w][(t * MB + m) * NB + n][r % 16][c % 16];
    }
    char* out = static_cast<char*>(p.out) + (int64_t)(loc.row + r) * p.out_row_bytes;
    float v = MODE == kGated ? gate(y[0], y[kMats - 1]) : y[0];
    if constexpr (MODE == kAdapted) {
      if (odd_values)
        v += odd_products<WD>(p, loc.row + r, row_pos[r] < 0 ? -1 : list[row_pos[r]], col);
    }
    if constexpr (MODE == kDense || MODE == kAdapted) {
      if (p.bias) v += load_elem(p.bias, col, WD);
      if (p.add) v += load_elem(out, col, p.out_dtype);
    }
    store_elem(out, col, p.out_dtype, v);
  }
}

}  // namespace dev
}  // namespace sgmv
