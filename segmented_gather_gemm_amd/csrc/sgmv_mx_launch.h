// sgmv_mx_launch.h -- interface between the entry points that quantise rows to
// microscaled 4-bit values and read them back (sgmv_mx_api.cpp) and their
// gfx950 kernels (sgmv_mx.hip).  Internal to libsgmv.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sgmv.h"
#include "sgmv_limits.h"

namespace sgmv {

struct MxParams {
  const void* in;          // quantise: rows of values; read back: null
  void* out;               // read back: rows of values
  void* codes;
  void* scales;
  const int64_t* rows;     // read back: row of codes for every row of out, or null
  int64_t row_bytes;       // of the values' rows
  int64_t code_stride;     // bytes
  int64_t scale_stride;
  int64_t R;               // read back: rows of codes
  uint32_t items;          // groups of 128 values over all rows
  uint32_t groups;         // of a row
  limits::Divisor by_groups;
  int32_t H;               // values of a row
  int32_t vec;             // 16-byte accesses are legal on whole blocks of eight values
};

constexpr int kMxThreads = 256;
constexpr int kMxUnroll = 2;                              // groups a lane works on
constexpr int kMxItems = kMxThreads / 16 * kMxUnroll;     // groups of a workgroup
constexpr int64_t kMxMaxItems = int64_t(1) << 28;         // a launch holds fewer than 2^32 threads
const void* mx_quantize_kernel(int xd);
const void* mx_dequantize_kernel(int od);

// Few tokens of a projection with adapters: the inputs' codes and scales (codes
// null: none) and the adapters' projections v = scale * x . lora_a^T in one
// launch.  A workgroup has one token and kMxProjectRows of a slice's rank.
struct MxProjectParams {
  const void* x;
  void* codes;
  void* scales;
  const int64_t* start;
  const int64_t* lens;
  const int64_t* idx;
  int64_t x_row_bytes;
  int64_t code_stride;
  int64_t scale_stride;
  int64_t T;
  int32_t H;               // a multiple of eight
  int32_t K;
  int32_t L;
  int32_t batches;
  int32_t parts;           // ceil(K / kMxProjectRows)
  int32_t v_stride;
  float scale;
  const void* a[SGMV_MAX_SLICES];  // lora_A (L, K, H) contiguous, 16-byte aligned
  float* v[SGMV_MAX_SLICES];       // (T, v_stride)
};
constexpr int kMxProjectWaves = 8, kMxProjectRows = kMxProjectWaves;
constexpr int kMxProjectAhead = 8;                        // blocks of eight values of a lane at a time
constexpr int kMxProjectStep = kMxProjectAhead * 64 * 8;  // values
const void* mx_project_kernel(int xd);

// Quantise the rows of `x` into codes and scales (shapes checked by the caller).
sgmv_status launch_mx_quantize(const sgmv_matrix& x, void* codes, int64_t code_stride, void* scales,
                               int64_t scale_stride, hipStream_t stream);

}  // namespace sgmv
