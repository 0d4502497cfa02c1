// Generic kernel of the shared projection with adapters and of the grouped
// products: any size, stride and alignment.
//
// A workgroup of four waves computes a tile of 64 rows x 64 output columns;
// wave w has 16 of the rows.  Operands go from global memory straight into
// matrix-instruction registers, 16 bytes a lane where rows are aligned and
// element by element where they are not.  Nothing is staged and every wave
// reads the tile's weights again (from the caches), so this kernel is bound
// by load latency; it is for the shapes that the tiled kernels do not take.
#include "sgmv_matmul.h"

namespace sgmv {
namespace dev {

template <int WD, bool GATED>
__global__ __launch_bounds__(kThreads) void matmul_generic(MatmulParams p) {
  __shared__ int32_t sh[kWaves + 4];
  __shared__ int32_t row_pos[kGenericRows], list[kGenericRows];
  __shared__ int32_t segs[adapter_words<kGenericRows>()], count[2], odd_found;
  constexpr int kBlocks = kGenericCols / 16;
  const TileLoc loc = find_tile<kThreads>(p, kGenericRows, sh);
  if (loc.row < 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n0 = loc.col * kGenericCols;
  const int row = loc.row + wave * 16 + (lane & 15);
  const bool live = row < loc.end;
  const int q = lane >> 4;  // which 8 of the 32 contraction steps this lane holds

  int64_t src = row;
  if (live && p.grouped && p.rows) src = p.rows[row];
  const bool have = live && src >= 0 && src < p.X;
  const char* xr = static_cast<const char*>(p.x) + (have ? src : 0) * p.x_row_bytes;
  const bool vx = ((reinterpret_cast<uintptr_t>(p.x) | (uint64_t)p.x_row_bytes) & 15) == 0;
  const char* wm = static_cast<const char*>(p.w) + (int64_t)loc.e * p.w_mat_bytes;
  const bool vw = ((reinterpret_cast<uintptr_t>(p.w) | (uint64_t)p.w_row_bytes |
                    (uint64_t)p.w_mat_bytes) & 15) == 0;

  f32x4 acc[GATED ? 2 : 1][kBlocks] = {};
  for (int h = 0; h < p.H; h += 32) {
    const int at = h + q * 8, cnt = clamp8((int64_t)p.H - at);
    u32x4 xv;
    load_any8<WD>(xr, at, have ? cnt : 0, vx, &xv);
#pragma unroll
    for (int f = 0; f < kBlocks; ++f) {
      const int n = n0 + f * 16 + (lane & 15);
#pragma unroll
      for (int g = 0; g < (GATED ? 2 : 1); ++g) {
        u32x4 wv;
        load_any8<WD>(wm + ((int64_t)g * p.N + (n < p.N ? n : 0)) * p.w_row_bytes, at,
                      n < p.N ? cnt : 0, vw, &wv);
        acc[g][f] = mfma<WD>(wv, xv, acc[g][f]);
      }
    }
  }

  bool odd_values = false;
  int32_t adapter = -1;  // of this lane's row
  if (!GATED && p.num_slices > 0) {
    if (threadIdx.x == 0) odd_found = 0;  // ahead of tile_adapters' barriers
    tile_adapters<kThreads, kGenericRows, false>(p, read_segment(p, threadIdx.x), loc.row, loc.end,
                                          row_pos, list, count, segs);
    const int32_t adapters = uniform(count[0]);
    const int32_t my_pos = row_pos[wave * 16 + (lane & 15)];
    for (int i = 0; i < adapters; ++i) {
      const int32_t a = uniform(list[i]);
      if (__ballot(my_pos == i) == 0) continue;  // none of this wave's rows
      // The sums go on from the accumulators and are kept in the lanes whose
      // token has the adapter.  float16 adds each step's products times 2^-e.
      f32x4 sum[kBlocks];
#pragma unroll
      for (int f = 0; f < kBlocks; ++f) sum[f] = acc[0][f];
      for (int s = 0; s < p.num_slices; ++s) {
        const AdapterDesc d = adapter_desc(s);
        if (d.offset >= n0 + kGenericCols || d.offset + d.n <= n0) continue;
        const bool vb = ((reinterpret_cast<uintptr_t>(d.b) & 15) == 0) && p.K % 8 == 0;
        for (int k = 0; k < p.K; k += 32) {
          const int at = k + q * 8, cnt = clamp8((int64_t)p.K - at);
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            v[j] = live && j < cnt ? d.v[(int64_t)row * p.v_stride + at + j] : 0.f;
          if (any_odd(v)) {
            drop_odd(v);
            if (my_pos >= 0) odd_found = 1;  // else no segment's row: anything may be there
          }
          int e = 0;
          if constexpr (WD == F16) {  // a token's 32 values are in four lanes
            e = split_exponent(quarters_max(largest_of(v)));
            scale_values(v, e);
          }
          u32x4 hi, lo;
          split_operand<WD>(v, &hi, &lo);
#pragma unroll
          for (int f = 0; f < kBlocks; ++f) {
            const int64_t n = (int64_t)n0 + f * 16 + (lane & 15) - d.offset;
            const bool in = n >= 0 && n < d.n;
            u32x4 bv;
            load_any8<WD>(d.b, ((int64_t)a * d.n + (in ? n : 0)) * p.K + at, in ? cnt : 0, vb, &bv);
            if (any_odd<WD>(bv)) {
              odd_found = 1;
              bv = drop_odd<WD>(bv);
            }
            f32x4 d = WD == F16 ? f32x4{} : sum[f];
            if (WD == BF16 && p.out_dtype == F32) d = mfma<WD>(bv, third_operand(v), d);
            d = mfma<WD>(bv, lo, d);
            d = mfma<WD>(bv, hi, d);
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[f][j] = WD == F16 ? sum[f][j] + ldexpf(d[j], -e) : d[j];
          }
        }
      }
#pragma unroll
      for (int f = 0; f < kBlocks; ++f)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[0][f][j] = my_pos == i ? sum[f][j] : acc[0][f][j];
    }
    __syncthreads();
    odd_values = uniform(odd_found) != 0;
    adapter = my_pos < 0 ? -1 : list[my_pos];
  }

  if (!live) return;
  char* orow = static_cast<char*>(p.out) + (int64_t)row * p.out_row_bytes;
#pragma unroll
  for (int f = 0; f < kBlocks; ++f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + f * 16 + q * 4 + i;
      if (n >= p.N) continue;
      float y;
      if constexpr (GATED) {
        y = gate(acc[0][f][i], acc[1][f][i]);
      } else {
        y = acc[0][f][i];
        if (odd_values) y += odd_products<WD>(p, row, adapter, n);
        if (p.bias) y += load_elem(p.bias, n, WD);
        if (p.add) y += load_elem(orow, n, p.out_dtype);
      }
      store_elem(orow, n, p.out_dtype, y);
    }
  }
}

}  // namespace dev

const void* matmul_generic_kernel(int wd, bool gated) {
  using namespace dev;
  if (wd == BF16)
    return gated ? (const void*)matmul_generic<BF16, true> : (const void*)matmul_generic<BF16, false>;
  if (wd == F16)
    return gated ? (const void*)matmul_generic<F16, true> : (const void*)matmul_generic<F16, false>;
  return nullptr;
}

}  // namespace sgmv
