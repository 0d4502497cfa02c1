// sgmv_mx_api.cpp -- libsgmv C entry points that quantise rows to microscaled
// 4-bit values (sgmv_mx_quantize) and read them back (sgmv_mx_dequantize):
// argument checks, sizing and launch.  No allocation, no synchronisation, no
// device-to-host traffic.
#include <stdint.h>

#include "sgmv.h"
#include "sgmv_host.h"
#include "sgmv_limits.h"
#include "sgmv_mx_host.h"
#include "sgmv_mx_launch.h"

namespace sgmv {

using namespace host;

namespace host {

sgmv_status check_mx(const sgmv_mx_stack& q, int64_t cols, const char* what) {
  const int64_t groups = limits::mx_groups(cols);
  if (q.num < 0 || q.rows < 0 || q.cols != cols || q.code_stride < groups * limits::kMxCodeBytes ||
      q.scale_stride < groups * limits::kMxScaleBytes)
    return fail(SGMV_ERR_INVALID_ARGUMENT,
                "%s: %lld x %lld rows of %lld values with strides %lld and %lld bytes do not hold "
                "rows of %lld values", what, (long long)q.num, (long long)q.rows, (long long)q.cols,
                (long long)q.code_stride, (long long)q.scale_stride, (long long)cols);
  if (q.code_stride % 16 != 0 || q.scale_stride % 4 != 0 || !aligned16(q.codes) ||
      (reinterpret_cast<uintptr_t>(q.scales) & 3) != 0)
    return fail(SGMV_ERR_INVALID_ARGUMENT,
                "%s: codes must be 16-byte aligned and scales 4-byte aligned, their strides too", what);
  return SGMV_OK;
}

}  // namespace host

namespace {

sgmv_status check_values(const sgmv_matrix& m, const char* what) {
  if (!known_dtype(m.dtype)) return fail(SGMV_ERR_INVALID_ARGUMENT, "unknown %s dtype %d", what, m.dtype);
  if (m.rows < 0 || m.cols < 1 || m.row_stride < m.cols)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "%s shape (%lld, %lld) with row stride %lld is invalid",
                what, (long long)m.rows, (long long)m.cols, (long long)m.row_stride);
  if (m.cols > INT32_MAX - 4096 || m.rows > kMxMaxItems / limits::mx_groups(m.cols))
    return fail(SGMV_ERR_UNSUPPORTED, "more than 2^28 groups of 128 values");
  return SGMV_OK;
}

MxParams params(const sgmv_matrix& m, void* codes, int64_t code_stride, void* scales,
                int64_t scale_stride) {
  MxParams p{};
  p.codes = codes;
  p.scales = scales;
  p.code_stride = code_stride;
  p.scale_stride = scale_stride;
  p.row_bytes = m.row_stride * elem_bytes(m.dtype);
  p.groups = (uint32_t)limits::mx_groups(m.cols);
  p.by_groups = limits::divisor(p.groups);
  p.items = (uint32_t)(m.rows * p.groups);
  p.H = (int32_t)m.cols;
  p.vec = aligned16(m.data) && p.row_bytes % 16 == 0;
  return p;
}

sgmv_status launch(const void* kernel, MxParams& p, hipStream_t stream) {
  void* args[] = {&p};
  const hipError_t e = hipLaunchKernel(kernel, dim3((p.items + kMxItems - 1) / kMxItems),
                                       dim3(kMxThreads), args, 0, stream);
  if (e != hipSuccess) return fail(SGMV_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  g_error.clear();
  return SGMV_OK;
}

}  // namespace

sgmv_status launch_mx_quantize(const sgmv_matrix& x, void* codes, int64_t code_stride, void* scales,
                               int64_t scale_stride, hipStream_t stream) {
  MxParams p = params(x, codes, code_stride, scales, scale_stride);
  p.in = x.data;
  return launch(mx_quantize_kernel(x.dtype), p, stream);
}

}  // namespace sgmv

extern "C" {

sgmv_status sgmv_mx_quantize(sgmv_matrix inputs, sgmv_mx_stack out, hipStream_t stream) {
  using namespace sgmv;
  sgmv_status st = check_values(inputs, "inputs");
  if (st != SGMV_OK) return st;
  st = check_mx(out, inputs.cols, "out");
  if (st != SGMV_OK) return st;
  if (out.num > INT32_MAX || out.rows > INT32_MAX || out.num * out.rows != inputs.rows)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "out must have the inputs' %lld rows", (long long)inputs.rows);
  if (inputs.rows == 0) {
    g_error.clear();
    return SGMV_OK;  // nothing to do
  }
  if (!inputs.data || !out.codes || !out.scales)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "null data pointer");
  return launch_mx_quantize(inputs, out.codes, out.code_stride, out.scales, out.scale_stride, stream);
}

sgmv_status sgmv_mx_dequantize(sgmv_mx_stack inputs, const int64_t* row_indices, sgmv_matrix out,
                               hipStream_t stream) {
  using namespace sgmv;
  sgmv_status st = check_values(out, "output");
  if (st != SGMV_OK) return st;
  st = check_mx(inputs, out.cols, "inputs");
  if (st != SGMV_OK) return st;
  if (inputs.num > INT32_MAX || inputs.rows > INT32_MAX)
    return fail(SGMV_ERR_UNSUPPORTED, "more than 2^31-1 rows or matrices");
  const int64_t rows = inputs.num * inputs.rows;
  if (!row_indices && rows != out.rows)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "output must have the inputs' %lld rows without row_indices",
                (long long)rows);
  if (out.rows == 0) {
    g_error.clear();
    return SGMV_OK;  // nothing to do
  }
  if (!out.data || (rows > 0 && (!inputs.codes || !inputs.scales)))
    return fail(SGMV_ERR_INVALID_ARGUMENT, "null data pointer");
  MxParams p = params(out, inputs.codes, inputs.code_stride, inputs.scales, inputs.scale_stride);
  p.out = out.data;
  p.rows = row_indices;
  p.R = rows;
  return launch(mx_dequantize_kernel(out.dtype), p, stream);
}

}  // extern "C"
