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
constexpr int kMxUnroll = 4;                              // groups a lane works on
constexpr int kMxItems = kMxThreads / 16 * kMxUnroll;     // groups of a workgroup
constexpr int64_t kMxMaxItems = int64_t(1) << 30;
const void* mx_quantize_kernel(int xd);
const void* mx_dequantize_kernel(int od);

// Quantise the rows of `x` into codes and scales (shapes checked by the caller).
sgmv_status launch_mx_quantize(const sgmv_matrix& x, void* codes, int64_t code_stride, void* scales,
                               int64_t scale_stride, hipStream_t stream);

}  // namespace sgmv
