// sgmv_route_api.cpp -- libsgmv C entry points of the expert routing
// (sgmv_route) and of the sum of a token's expert rows (sgmv_combine):
// argument checks, sizing and launch.  No allocation, no synchronisation, no
// device-to-host traffic.
#include <stdint.h>

#include "sgmv.h"
#include "sgmv_host.h"
#include "sgmv_route_launch.h"

namespace {

using namespace sgmv::host;

static_assert(SGMV_MAX_EXPERTS == sgmv::kRouteMaxExperts && SGMV_MAX_TOP_K == sgmv::kRouteMaxTopK,
              "public limits");

// Workgroups of a routing call and the tokens of each: rounds of up to
// kRouteEntries choices, at most kRouteMaxBlocks workgroups.
void route_split(int64_t T, int64_t k, int64_t* blocks, int64_t* block_tokens,
                 int64_t* round_tokens) {
  int64_t round = sgmv::kRouteEntries / k;
  if (round > 128) round = 128;
  int64_t per = (T + sgmv::kRouteMaxBlocks - 1) / sgmv::kRouteMaxBlocks;
  if (per < round) per = round;
  *blocks = (T + per - 1) / per;
  *block_tokens = per;
  *round_tokens = round;
}

sgmv_status check_route(int64_t tokens, int64_t experts, int64_t top_k) {
  if (tokens < 0 || experts < 1 || top_k < 1 || top_k > experts)
    return fail(SGMV_ERR_INVALID_ARGUMENT,
                "routing needs tokens >= 0 and 1 <= top_k <= experts, got %lld, %lld, %lld",
                (long long)tokens, (long long)top_k, (long long)experts);
  if (experts > SGMV_MAX_EXPERTS || top_k > SGMV_MAX_TOP_K)
    return fail(SGMV_ERR_UNSUPPORTED, "more than %d experts or %d choices", SGMV_MAX_EXPERTS,
                SGMV_MAX_TOP_K);
  if (tokens > (1 << 30) / top_k)
    return fail(SGMV_ERR_UNSUPPORTED, "more than 2^30 choices (tokens x top_k)");
  return SGMV_OK;
}

size_t route_bytes(int64_t tokens, int64_t experts, int64_t top_k) {
  int64_t blocks, per, round;
  route_split(tokens, top_k, &blocks, &per, &round);
  return blocks > 1 ? (size_t)(blocks * experts * 4) : 0;
}

}  // namespace

extern "C" {

sgmv_status sgmv_route_workspace_bytes(int64_t tokens, int64_t experts, int64_t top_k,
                                       size_t* bytes) {
  if (!bytes) return fail(SGMV_ERR_INVALID_ARGUMENT, "bytes pointer is null");
  const sgmv_status st = check_route(tokens, experts, top_k);
  if (st != SGMV_OK) return st;
  *bytes = route_bytes(tokens, experts, top_k);
  g_error.clear();
  return SGMV_OK;
}

sgmv_status sgmv_route(sgmv_matrix logits, int64_t top_k, int renormalize, float* weights,
                       int64_t* experts, int64_t* slots, int64_t* row_indices,
                       int64_t* b_seq_start_loc, int64_t* seq_lens, void* workspace,
                       size_t workspace_bytes, hipStream_t stream) {
  using namespace sgmv;
  if (!known_dtype(logits.dtype))
    return fail(SGMV_ERR_INVALID_ARGUMENT, "unknown logits dtype %d", logits.dtype);
  if (logits.row_stride < logits.cols)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "logits' row stride %lld is below their %lld columns",
                (long long)logits.row_stride, (long long)logits.cols);
  sgmv_status st = check_route(logits.rows, logits.cols, top_k);
  if (st != SGMV_OK) return st;
  if (!b_seq_start_loc || !seq_lens)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "segment metadata pointer is null");
  if (logits.rows > 0 && (!logits.data || !weights || !experts || !slots || !row_indices))
    return fail(SGMV_ERR_INVALID_ARGUMENT, "null data pointer");
  const size_t need = route_bytes(logits.rows, logits.cols, top_k);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned16(workspace)))
    return fail(SGMV_ERR_INVALID_ARGUMENT,
                "workspace must be 16-byte aligned and hold %zu bytes, got %zu", need,
                workspace ? workspace_bytes : (size_t)0);

  RouteParams p{};
  p.logits = logits.data;
  p.weights = weights;
  p.experts = experts;
  p.slots = slots;
  p.rows = row_indices;
  p.start = b_seq_start_loc;
  p.lens = seq_lens;
  p.counts = static_cast<int32_t*>(workspace);
  p.logits_row_bytes = logits.row_stride * elem_bytes(logits.dtype);
  p.T = (int32_t)logits.rows;
  p.E = (int32_t)logits.cols;
  p.k = (int32_t)top_k;
  p.dtype = logits.dtype;
  p.renormalize = renormalize != 0;
  p.vec = p.E % route_lane_experts(p.E) == 0 && aligned16(logits.data) &&
          p.logits_row_bytes % 16 == 0;
  int64_t blocks, per, round;
  route_split(logits.rows, top_k, &blocks, &per, &round);
  if (blocks < 1) blocks = 1;  // no token: the empty segments are still written
  p.blocks = (int32_t)blocks;
  p.block_tokens = (int32_t)per;
  p.round_tokens = (int32_t)round;
  void* args[] = {&p};
  const size_t lds = (size_t)p.E * 4 * (1 + kRouteThreads / 64);
  hipError_t e = hipLaunchKernel(route_select_kernel(p.E), dim3((unsigned)blocks),
                                 dim3(kRouteThreads), args, lds, stream);
  if (e == hipSuccess && blocks > 1)
    e = hipLaunchKernel(route_place_kernel(), dim3((unsigned)blocks), dim3(kRouteThreads), args,
                        (size_t)p.E * 8, stream);
  if (e != hipSuccess) return fail(SGMV_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  g_error.clear();
  return SGMV_OK;
}

sgmv_status sgmv_combine(sgmv_matrix rows, const float* weights, const int64_t* slots,
                         int64_t top_k, sgmv_matrix out, int add_inputs, hipStream_t stream) {
  using namespace sgmv;
  if (!known_dtype(rows.dtype) || !known_dtype(out.dtype))
    return fail(SGMV_ERR_INVALID_ARGUMENT, "unknown dtype");
  if (rows.rows < 0 || rows.cols < 0 || rows.row_stride < rows.cols)
    return fail(SGMV_ERR_INVALID_ARGUMENT, "rows shape (%lld, %lld) with row stride %lld is invalid",
                (long long)rows.rows, (long long)rows.cols, (long long)rows.row_stride);
  if (out.rows < 0 || out.cols != rows.cols || out.row_stride < out.cols)
    return fail(SGMV_ERR_INVALID_ARGUMENT,
                "output (%lld, %lld) with row stride %lld must have the rows' %lld columns",
                (long long)out.rows, (long long)out.cols, (long long)out.row_stride,
                (long long)rows.cols);
  if (top_k < 0) return fail(SGMV_ERR_INVALID_ARGUMENT, "top_k must be >= 0");
  if (rows.cols > INT32_MAX - 8 || top_k > INT32_MAX || out.rows > INT32_MAX)
    return fail(SGMV_ERR_UNSUPPORTED, "more than 2^31-1 rows, columns or choices");
  if (out.rows == 0 || out.cols == 0) {
    g_error.clear();
    return SGMV_OK;  // nothing to do
  }
  if (!out.data || (rows.rows > 0 && !rows.data))
    return fail(SGMV_ERR_INVALID_ARGUMENT, "null data pointer");
  if (top_k > 0 && (!weights || !slots))
    return fail(SGMV_ERR_INVALID_ARGUMENT, "weights or slots pointer is null");

  CombineParams p{};
  p.rows = rows.data;
  p.weights = weights;
  p.slots = slots;
  p.out = out.data;
  p.rows_row_bytes = rows.row_stride * elem_bytes(rows.dtype);
  p.out_row_bytes = out.row_stride * elem_bytes(out.dtype);
  p.R = rows.rows;
  p.T = out.rows;
  p.H = (int32_t)rows.cols;
  p.k = (int32_t)top_k;
  p.out_dtype = out.dtype;
  p.add = add_inputs != 0;
  p.vec = p.H % 8 == 0 && aligned16(rows.data) && aligned16(out.data) &&
          p.rows_row_bytes % 16 == 0 && p.out_row_bytes % 16 == 0;
  const int64_t work = p.T * ((p.H + 7) / 8);
  const int64_t most = 256 * 8 * 4;
  int64_t grid = (work + kCombineThreads - 1) / kCombineThreads;
  if (grid > most) grid = most;
  void* args[] = {&p};
  const hipError_t e = hipLaunchKernel(combine_kernel(rows.dtype), dim3((unsigned)grid),
                                       dim3(kCombineThreads), args, 0, stream);
  if (e != hipSuccess) return fail(SGMV_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(e));
  g_error.clear();
  return SGMV_OK;
}

}  // extern "C"
