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
  u32x4 wv[2][G][kMats][NB][2], xv[2][G][MB][2];
  f32x4 acc[kMats][MB][NB] = {};
  auto load = [&](int buf, int u) __attribute__((always_inline)) {
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int k = (wave + (u + g) * kW) * 64 + s * 32 + lq * 8;
        const bool in = u + g < mine && k < p.H;
#pragma unroll
        for (int t = 0; t < kMats; ++t)
#pragma unroll
          for (int n = 0; n < NB; ++n)
            buf_load8<WD>(wr[t], in ? woff[n] + k * 2u : kOut, &wv[buf][g][t][n][s]);
#pragma unroll
        for (int m = 0; m < MB; ++m)
          buf_load8<WD>(xr, in ? xoff[m] + k * 2u : kOut, &xv[buf][g][m][s]);
      }
  };
  auto use = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int t = 0; t < kMats; ++t)
#pragma unroll
          for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int n = 0; n < NB; ++n)
              acc[t][m][n] = mfma<WD>(wv[buf][g][t][n][s], xv[buf][g][m][s], acc[t][m][n]);
  };
  load(0, 0);
  for (int u = 0; u < mine; u += 2 * G) {
    load(1, u + G);
    use(0);
    load(0, u + 2 * G);
    use(1);
  }

  // Adapters, one after another dealt to the waves: each wave's products go
  // to the lanes whose token has the adapter, so that what one request's
  // weights hold never reaches another's rows.
  if constexpr (MODE == kAdapted) {
    __shared__ int32_t row_a[ROWS], list[ROWS], segs[3 * ROWS], count[2];
    tile_adapters<kNT, ROWS>(p, read_segment(p, threadIdx.x), loc.row, loc.end, row_a, list, count,
                             segs);
    const int adapters = uniform(count[0]);
    for (int i = wave; i < adapters; i += kW) {
      const int a = uniform(list[i]);
      f32x4 d[MB][NB] = {};
      for (int sl = 0; sl < p.num_slices; ++sl) {
        const AdapterDesc ad = adapter_desc(sl);
        if (ad.offset >= n0 + 16 * NB || ad.offset + ad.n <= n0) continue;
        const rsrc_t br = uniform_rsrc(static_cast<const char*>(ad.b) + a * ad.n * p.K * 2,
                                       ad.n * p.K * 2);
        const rsrc_t vr =
            uniform_rsrc(reinterpret_cast<const char*>(ad.v + (int64_t)loc.row * p.v_stride),
                         (int64_t)rows * p.v_stride * 4);
        for (int k = 0; k < p.K; k += 32) {
          const int at = k + lq * 8;
          u32x4 bv[NB], hi[MB], lo[MB];
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            const int c = n0 + n * 16 + lr - (int)ad.offset;
            buf_load8<WD>(br, c >= 0 && c < ad.n && at < p.K ? (uint32_t)(c * p.K + at) * 2u : kOut,
                          &bv[n]);
          }
#pragma unroll
          for (int m = 0; m < MB; ++m) {
            u32x4 raw[2];
            buf_load8<F32>(vr, at < p.K ? (uint32_t)((m * 16 + lr) * p.v_stride + at) * 4u : kOut,
                           raw);
            float v[8];
            out_values<F32>(raw, v);
            split_operand<WD>(v, &hi[m], &lo[m]);
          }
#pragma unroll
          for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int n = 0; n < NB; ++n) {
              d[m][n] = mfma<WD>(bv[n], hi[m], d[m][n]);
              d[m][n] = mfma<WD>(bv[n], lo[m], d[m][n]);
            }
        }
      }
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        const bool own = row_a[m * 16 + lr] == a;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[0][m][n][j] += own ? d[m][n][j] : 0.f;
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
    if constexpr (MODE == kDense || MODE == kAdapted) {
      if (p.bias) v += load_elem(p.bias, col, WD);
      if (p.add) v += load_elem(out, col, p.out_dtype);
    }
    store_elem(out, col, p.out_dtype, v);
  }
}

template <int WD, int MB, int NB, int G>
const void* skinny_kernel(int mode) {
  switch (mode) {
    case kDense: return (const void*)matmul_skinny<WD, kDense, MB, NB, G>;
    case kGrouped: return (const void*)matmul_skinny<WD, kGrouped, MB, NB, G>;
    case kGated:
      if constexpr (MB * NB < 8) return (const void*)matmul_skinny<WD, kGated, MB, NB, G>;
      return nullptr;
    default: return (const void*)matmul_skinny<WD, kAdapted, MB, NB, G>;
  }
}

}  // namespace dev
}  // namespace sgmv
