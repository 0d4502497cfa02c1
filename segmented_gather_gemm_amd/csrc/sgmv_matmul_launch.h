// sgmv_matmul_launch.h -- interface between the entry points of the shared
// projection with adapters and of the grouped products
// (sgmv_matmul_api.cpp) and their gfx950 kernels (sgmv_matmul_*.hip).
// Internal to libsgmv.
#pragma once

#include "sgmv_launch.h"

namespace sgmv {

// One adapter slice: y[t][offset + n] += sum_k v[t][k] * b[a][n][k].
struct AdapterDesc {
  const void* b;        // lora_B (L, n, K) contiguous
  const float* v;       // projected rows (T, K) float32, scale applied, row stride v_stride
  int64_t n;            // slice width
  int64_t offset;       // first output column
};

// Products out[t][n] = sum_h x[src(t)][h] * w[e][n][h].  Two layouts:
//  * dense (grouped == 0): one weight matrix, every row of out, plus the
//    adapters of the segments' rows (start, lens, idx);
//  * grouped: the rows of segment b with weight matrix idx[b] (idx null: b).
// The segment fields keep Params' names.
struct MatmulParams {
  const void* x;
  const void* w;
  const void* bias;       // dense: (N) of the weights' dtype, or null
  void* out;
  const int64_t* start;
  const int64_t* lens;
  const int64_t* idx;
  const int64_t* rows;    // grouped: row of x for every row of out, or null
  int64_t x_row_bytes;
  int64_t w_row_bytes;
  int64_t w_mat_bytes;    // bytes from one weight matrix to the next
  int64_t out_row_bytes;
  int64_t T;              // rows of out
  int64_t X;              // rows of x
  int32_t H;              // contraction length
  int32_t N;              // output columns (gated: half of a weight matrix's rows)
  int32_t batches;
  int32_t L;              // weight matrices (dense: adapters)
  int32_t grouped;
  int32_t out_dtype;
  int32_t add;            // dense: accumulate onto out
  int32_t vec_out;        // out's rows are 16-byte aligned and its columns a multiple of eight
  int32_t col_tiles;      // column tiles of the launch
  int32_t row_tiles;      // dense: row tiles; grouped: bound on them (the device counts)
  int32_t num_slices;     // adapters: slices, rank, v's row stride (floats)
  int32_t K;
  int32_t v_stride;
  AdapterDesc s[kMaxSlices];
};

// Generic kernel: any size, stride and alignment (64 x 64 tiles).
constexpr int kGenericRows = 64, kGenericCols = 64;
const void* matmul_generic_kernel(int wd, bool gated);

// Tiled kernels: rows of 16-byte blocks (hidden a multiple of eight, 16-byte
// aligned rows of x and w) that 32-bit offsets reach.  mode: 0 dense, 1
// grouped, 2 gated, 3 dense with adapters.
struct TiledKernel {
  const void* kernel;
  int rows, cols, threads;  // of a tile, of a workgroup
};
TiledKernel matmul_tiled_large(int wd, int mode);
TiledKernel matmul_tiled_medium(int wd, int mode);
// Few rows (the same requirements): tiles of 16 rows, of 32 for dense calls
// and of 64 for dense calls with adapters.
TiledKernel matmul_skinny_16(int wd, int mode);
TiledKernel matmul_skinny_32(int wd, bool adapted);
TiledKernel matmul_skinny_64_adapted(int wd);

}  // namespace sgmv
