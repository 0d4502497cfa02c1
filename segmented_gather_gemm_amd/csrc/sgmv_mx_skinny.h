// sgmv_mx_skinny.h -- gfx950 kernel of the shared projection with adapters and
// of the grouped products with microscaled 4-bit weights for few rows (decode
// batches, single tokens).  Internal to libsgmv.
//
// A few rows against a whole weight matrix are bound by reading the weights
// once.  A workgroup of eight waves keeps its 16 MB input rows in registers
// and walks over tiles of 16 weight rows (output columns); the contraction is
// dealt to the waves in chunks of two groups (256 values, 128 bytes of codes a
// row), chunk c to wave c mod 8.  Up to 16 rows are quantised here: a lane's share
// of a matrix instruction's input rows is one whole block of 32 values of one
// row, so that this needs no exchange between lanes.  Loads of the next tile are
// in flight while a tile's eight partial sums meet in LDS and are added in order
// (two sets of them, one barrier a tile).
//
// Adapters: each result's part is summed in float32 on the vector unit, a row
// with its own adapter, in order of k: for the few rows of a decode batch that is
// less than gathering the rows of each adapter for the matrix unit.  One or two
// tokens' projections are made here as well.
//
// Measured, hidden 4096, bfloat16: 4096 columns, one token 6.8 us, with its
// adapter of rank 16 10.2-10.5 (of which 3.4 its projection, a chain of two loads from
// memory and a sum over the wave; a launch of its own takes 4.5 and the gap);
// 28672 columns (62 MB of codes and scales), 1 and 16 rows 15.4 and 17.7 us, 4.0
// and 3.5 TB/s; 64 rows of 32 adapters, QKV's 6144 columns, 13.2-13.7 us, of which reading
// the weights would take 2.6: bound by latency.  A workgroup has three tiles here, the
// weights of one ahead, and as loads arrive in order, a tile's lora_B arrives
// behind the next tile's weights.
#pragma once

#include "sgmv_matmul.h"
#include "sgmv_mx.h"
#include "sgmv_mx_launch.h"

namespace sgmv {
namespace dev {

// Fill adapter[0 .. ROWS) with the adapters of rows row0 .. end (-1: none; all
// NT threads take part).  Segments are disjoint.
template <int NT, int ROWS>
__device__ __forceinline__ void row_adapters(const MatmulParams& p, Segment seg, int32_t row0,
                                             int32_t end, int32_t* adapter) {
  const int tid = threadIdx.x;
  if (tid < ROWS) adapter[tid] = -1;
  __syncthreads();
  for (int32_t b = tid; b < p.batches; b += NT) {
    if (b >= NT) seg = read_segment(p, b);
    const int64_t st = seg.start, ln = seg.len, a = seg.a;
    if (a < 0 || a >= p.L || ln <= 0 || st < 0 || st > p.T - ln) continue;
    const int64_t from = st > row0 ? st : row0, to = st + ln < end ? st + ln : end;
    for (int64_t r = from; r < to; ++r) adapter[r - row0] = (int32_t)a;
  }
  __syncthreads();
}

// sum_k v(row, s)[k] b[a][n][k] over the slice s that holds column n, in order of k
// (0 without an adapter or such a slice).  Whole blocks of eight, aligned.
template <int WD, class V>
__device__ __forceinline__ float adapter_product(const MatmulParams& p, int32_t a, int n, V v_of) {
  float sum = 0.f;
  for (int s = 0; s < p.num_slices; ++s) {
    const AdapterDesc d = adapter_desc(s);
    if (a < 0 || n < d.offset || n >= d.offset + d.n) continue;
    const int64_t at = ((int64_t)a * d.n + n - d.offset) * p.K;
    const float* vr = v_of(d, s);
#pragma unroll 2
    for (int k = 0; k < p.K; k += 8) {
      u32x4 bv, raw[2];
      load_vec8<WD>(d.b, at + k, &bv);
      load_vec8<F32>(vr, k, raw);
      float b[8], v[8];
      out_values<WD>(&bv, b);
      out_values<F32>(raw, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(v[j], b[j], sum);
    }
  }
  return sum;
}

// projected[row][slice][k] = scale * x[row] . lora_A[adapter][k] for the slices that
// this workgroup's columns are in: a wave two k at a time (four: one token's
// QKV 16.4 against 14.9 us), lora_A (in v's place) and x in blocks of eight a
// lane; the order of a sum is mx_project's.  Every workgroup does that for itself.
template <int WD>
__device__ __forceinline__ void project_rows(const MatmulParams& p, const TileLoc& loc, int tiles,
                                             const int32_t* adapter, float* projected) {
  constexpr int R = 2;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int count = (loc.end - loc.row) * p.num_slices * p.K;
  for (int i = R * wave; i < count; i += R * kMxSkinnyWaves) {
    const int rs = i / p.K, k = i - rs * p.K, r = rs / p.num_slices;
    const AdapterDesc d = adapter_desc(rs - r * p.num_slices);
    const int a = uniform(adapter[r]);
    bool used = false;
    for (int tile = loc.col; tile < tiles; tile += p.col_tiles)
      used = used || (tile * 16 < d.offset + d.n && tile * 16 + 16 > d.offset);
    if (a < 0 || !used) continue;
    const char* x = static_cast<const char*>(p.x) + (loc.row + r) * p.x_row_bytes;
    const char* la = reinterpret_cast<const char*>(d.v) + ((int64_t)a * p.K + k) * p.mx_hidden * 2;
    float sum[R] = {};
    for (int base = 0; base < p.mx_hidden; base += kMxProjectStep) {
      u32x4 xv[kMxProjectAhead], av[R][kMxProjectAhead];
#pragma unroll
      for (int j = 0; j < kMxProjectAhead; ++j) {
        const int64_t at = base + (j * 64 + lane) * 8;
        const bool in = at < p.mx_hidden;
        xv[j] = in ? *reinterpret_cast<const u32x4*>(x + at * 2) : u32x4{};
#pragma unroll
        for (int h = 0; h < R; ++h)
          av[h][j] = in ? *reinterpret_cast<const u32x4*>(la + (h * (int64_t)p.mx_hidden + at) * 2) : u32x4{};
      }
#pragma unroll
      for (int j = 0; j < kMxProjectAhead; ++j) {
        float xf[8], f[8];
        out_values<WD>(&xv[j], xf);
#pragma unroll
        for (int h = 0; h < R; ++h) {
          out_values<WD>(&av[h][j], f);
#pragma unroll
          for (int q = 0; q < 8; ++q) sum[h] = fmaf(xf[q], f[q], sum[h]);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < R; ++h) {
      const float v = wave_sum(sum[h]) * p.scale;
      if (lane == 0) projected[i + h] = v;
    }
  }
}

// C: chunks of a wave that it holds at a time; longer contractions take several
// such sets (and read their inputs again for each tile).
template <int WD, int MODE, int MB, int C>
__global__ __launch_bounds__(64 * kMxSkinnyWaves, 2) void mx_skinny_rows(MatmulParams p) {
  constexpr int kW = kMxSkinnyWaves, kNT = 64 * kW, ROWS = 16 * MB;
  constexpr int kMats = MODE == kGated ? 2 : 1;  // weight blocks of a tile
  constexpr int kBlocks = MB * kMats, kPad = 20;
  constexpr bool kQuantise = MB == 1;  // else x comes as codes and scales
  __shared__ int32_t sh[kW + 4];
  __shared__ float part[2][kW][kBlocks][16][kPad];
  __shared__ int32_t row_adapter[MODE == kAdapted ? ROWS : 1];
  constexpr bool kProjects = kQuantise && MODE == kAdapted;
  __shared__ __attribute__((aligned(16))) float projected[kProjects ? kMxProjectMost : 1];
  const TileLoc loc = find_tile<kNT>(p, ROWS, sh);
  if (loc.row < 0) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int rows = loc.end - loc.row;
  const int lr = lane & 15, lq = lane >> 4;

  const bool gather = (MODE == kGrouped || MODE == kGated) && p.rows != nullptr;
  const rsrc_t xr =
      uniform_rsrc(static_cast<const char*>(p.x) + (gather ? 0 : loc.row) * p.x_row_bytes,
                   ((gather ? p.X : rows) - 1) * p.x_row_bytes +
                       (int64_t)(kQuantise ? p.mx_hidden : p.H) * 2);
  rsrc_t xsr = xr;
  if constexpr (!kQuantise)
    xsr = uniform_rsrc(static_cast<const char*>(p.xs) + loc.row * p.xs_row_bytes,
                       (rows - 1) * p.xs_row_bytes + p.H / 8);
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

  const int groups = p.H / 32, chunks = (groups + 1) / 2;
  const int sets = (chunks + kW * C - 1) / (kW * C);
  const int tiles = (p.N + 15) / 16, step = p.col_tiles;

  // Set s's inputs: codes and scales of the lane's blocks.
  u32x4 xv[MB][C][2];
  uint32_t xs[MB][C][2];
  auto read_x = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int g = ((s * C + c) * kW + wave) * 2;
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        if constexpr (kQuantise) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int at = (g + h) * 128 + lq * 32;
            u32x4 raw[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              buf_load8<WD>(xr, at + i * 8 < p.mx_hidden ? xoff[m] + (uint32_t)(at + i * 8) * 2u : kOut, &raw[i]);
            xs[m][c][h] = mx_scale(mx_largest<WD>(raw));
#pragma unroll
            for (int i = 0; i < 4; ++i) xv[m][c][h][i] = mx_codes8<WD>(&raw[i], xs[m][c][h]);
          }
        } else {
          const int r = m * 16 + lr;  // rows past the tile's end pass the resources'
#pragma unroll
          for (int h = 0; h < 2; ++h)
            buf_load8<WD>(xr, g + h < groups ? (uint32_t)(r * p.x_row_bytes + (g + h) * 64 + lq * 16) : kOut,
                          &xv[m][c][h]);
          const uint2 w = __builtin_bit_cast(
              uint2, __builtin_amdgcn_raw_buffer_load_b64(
                         xsr, (int)(g < groups ? (uint32_t)(r * p.xs_row_bytes + g * 4) : kOut), 0, 0));
          xs[m][c][0] = w.x >> (8 * lq);
          xs[m][c][1] = g + 1 < groups ? w.y >> (8 * lq) : 0u;  // an odd row's last word is the next row's
        }
      }
    }
  };

  // A tile's weights of set s: 16 rows' codes, and the two words of scales of
  // each chunk, a byte of which is the lane's.
  u32x4 wv[kMats][C][2];
  uint2 ws[kMats][C];
  auto read_w = [&](int tile, int s) __attribute__((always_inline)) {
    const int n0 = tile * 16;
    const int64_t nr = p.N - n0 < 16 ? p.N - n0 : 16;  // none past the last tile
#pragma unroll
    for (int t = 0; t < kMats; ++t) {
      const int64_t first = limits::stack_row(loc.e, kMats * (int64_t)p.N, t * (int64_t)p.N + n0);
      const rsrc_t wr = uniform_rsrc(static_cast<const char*>(p.w) + first * p.w_row_bytes,
                                     nr <= 0 ? 0 : (nr - 1) * p.w_row_bytes + (int64_t)p.H * 2);
      const rsrc_t sr = uniform_rsrc(static_cast<const char*>(p.ws) + first * p.ws_row_bytes,
                                     nr <= 0 ? 0 : (nr - 1) * p.ws_row_bytes + p.H / 8);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int g = ((s * C + c) * kW + wave) * 2;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          buf_load8<WD>(wr, g + h < groups ? (uint32_t)(lr * p.w_row_bytes + (g + h) * 64 + lq * 16) : kOut,
                        &wv[t][c][h]);
        ws[t][c] = __builtin_bit_cast(
            uint2, __builtin_amdgcn_raw_buffer_load_b64(
                       sr, (int)(g < groups ? (uint32_t)(lr * p.ws_row_bytes + g * 4) : kOut), 0, 0));
      }
    }
  };

  Segment seg{};
  if constexpr (MODE == kAdapted) seg = read_segment(p, threadIdx.x);
  read_w(loc.col, 0);
  if constexpr (MODE == kAdapted)
    row_adapters<kNT, ROWS>(p, seg, loc.row, loc.end, row_adapter);
  if constexpr (kProjects) {
    if (p.projects) {
      project_rows<WD>(p, loc, tiles, row_adapter, projected);
      __syncthreads();
    }
  }

  constexpr int kMine = (ROWS * 16 + kNT - 1) / kNT;  // results of a thread in a tile
  int buffer = 0;
  for (int tile = loc.col; tile < tiles; tile += step, buffer ^= 1) {
    f32x4 acc[kMats][MB] = {};
    for (int s = 0; s < sets; ++s) {
      if (sets > 1 || tile == loc.col) read_x(s);
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int t = 0; t < kMats; ++t) {
            const bool in = ((s * C + c) * kW + wave) * 2 + h < groups;
            const uint32_t sw = in ? (h == 0 ? ws[t][c].x : ws[t][c].y) >> (8 * lq) : 0u;
#pragma unroll
            for (int m = 0; m < MB; ++m)
              acc[t][m] = mfma_fp4<0>(wv[t][c][h], xv[m][c][h], acc[t][m], sw, xs[m][c][h]);
          }
      const bool last = s + 1 == sets;
      read_w(last ? tile + step : tile, last ? 0 : s + 1);
    }
#pragma unroll
    for (int t = 0; t < kMats; ++t)
#pragma unroll
      for (int m = 0; m < MB; ++m)
        *reinterpret_cast<f32x4*>(&part[buffer][wave][t * MB + m][lr][lq * 4]) = acc[t][m];
    [[maybe_unused]] float extra[kMine];
    if constexpr (MODE == kAdapted) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int e = threadIdx.x + i * kNT, r = e / 16;
        extra[i] = 0.f;
        if (r >= rows) continue;
        const int a = row_adapter[r], n = tile * 16 + e % 16;
        if (kProjects && p.projects)
          extra[i] = adapter_product<WD>(p, a, n, [&](const AdapterDesc&, int s) {
            return &projected[(r * p.num_slices + s) * p.K];
          });
        else
          extra[i] = adapter_product<WD>(p, a, n, [&](const AdapterDesc& d, int) {
            return d.v + (int64_t)(loc.row + r) * p.v_stride;
          });
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int e = threadIdx.x + i * kNT, r = e / 16, col = tile * 16 + e % 16;
      if (r >= rows || col >= p.N) continue;
      float y[kMats];
#pragma unroll
      for (int t = 0; t < kMats; ++t) {
        y[t] = 0.f;
#pragma unroll
        for (int w = 0; w < kW; ++w) y[t] += part[buffer][w][t * MB + r / 16][r % 16][e % 16];
      }
      char* out = static_cast<char*>(p.out) + (int64_t)(loc.row + r) * p.out_row_bytes;
      float v = MODE == kGated ? gate(y[0], y[kMats - 1]) : y[0];
      if constexpr (MODE == kAdapted) v += extra[i];
      if constexpr (MODE == kDense || MODE == kAdapted) {
        if (p.bias) v += load_elem(p.bias, col, WD);
        if (p.add) v += load_elem(out, col, p.out_dtype);
      }
      store_elem(out, col, p.out_dtype, v);
    }
  }
}

}  // namespace dev
}  // namespace sgmv
