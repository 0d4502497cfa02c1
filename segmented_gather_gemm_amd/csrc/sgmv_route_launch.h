// sgmv_route_launch.h -- interface between the entry points of the expert
// routing and of the sum of a token's expert rows (sgmv_route_api.cpp) and
// their gfx950 kernels (sgmv_route.hip).  Internal to libsgmv.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sgmv {

constexpr int kRouteThreads = 512;
constexpr int kRouteEntries = 512;    // (token, choice) pairs of one round of a workgroup
constexpr int kRouteMaxBlocks = 256;  // workgroups of a call: their expert counts are read by all
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopK = 32;

struct RouteParams {
  const void* logits;     // (T, E), row stride in bytes
  float* weights;         // (T, k)
  int64_t* experts;       // (T, k)
  int64_t* slots;         // (T, k)
  int64_t* rows;          // (T k)
  int64_t* start;         // (E)
  int64_t* lens;          // (E)
  int32_t* counts;        // (blocks, E) expert counts, when blocks > 1
  int64_t logits_row_bytes;
  int32_t T, E, k;
  int32_t dtype;
  int32_t renormalize;
  int32_t vec;            // rows aligned for loads of a lane's experts, which divide E
  int32_t blocks;
  int32_t block_tokens;   // tokens of a workgroup
  int32_t round_tokens;   // tokens of a round: round_tokens * k <= kRouteEntries
};

// Selection kernel for E experts, and the kernel that places the choices
// (calls of more than one workgroup).
const void* route_select_kernel(int experts);
int route_lane_experts(int experts);  // consecutive experts a lane of it holds
const void* route_place_kernel();

struct CombineParams {
  const void* rows;       // (R, H)
  const float* weights;   // (T, k)
  const int64_t* slots;   // (T, k)
  void* out;              // (T, H)
  int64_t rows_row_bytes;
  int64_t out_row_bytes;
  int64_t R;
  int64_t T;
  int32_t H, k;
  int32_t out_dtype;
  int32_t add;
  int32_t vec;            // 16-byte accesses are legal and H % 8 == 0
};

constexpr int kCombineThreads = 256;
const void* combine_kernel(int dtype);

}  // namespace sgmv
