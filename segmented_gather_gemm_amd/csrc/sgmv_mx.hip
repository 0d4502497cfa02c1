// Kernels that quantise rows to microscaled 4-bit values and read them back.
//
// A lane has eight values (16 bytes of 16-bit ones), four lanes a block of 32,
// sixteen lanes a group of 128: the block's largest magnitude takes two
// exchanges inside a quad of lanes, loads and stores are consecutive over the
// lanes, and a group's four scale bytes leave as one word.  Groups are dealt to
// the lanes over all rows, whatever a row's length, kMxUnroll of them a lane so
// that several loads are in flight.  Bound by memory.
#include "sgmv_mx.h"
#include "sgmv_mx_launch.h"

namespace sgmv {
namespace dev {

// A lane's value with what DPP control CTRL (of all lanes' exchange) brings it.
template <int CTRL>
__device__ __forceinline__ uint32_t from_lane(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kRowRor4 = 0x124, kRowRor8 = 0x128;

__device__ __forceinline__ uint32_t first_item() {
  return blockIdx.x * kMxItems + (threadIdx.x >> 6) * 4 * kMxUnroll + ((threadIdx.x & 63) >> 4);
}

template <int XD>
__global__ __launch_bounds__(kMxThreads) void mx_quantize(MxParams p) {
  constexpr int U = kMxUnroll;
  const int lane = threadIdx.x & 15;  // of the group
  u32x4 raw[U][raw_vecs<XD>()];
  uint32_t row[U], g[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t item = first_item() + u * 4;
    const bool ok = item < p.items;
    row[u] = ok ? limits::divide(item, p.by_groups) : 0;
    g[u] = item - row[u] * p.groups;
    const int64_t at = (int64_t)g[u] * 128 + lane * 8;
    load_any8<XD>(static_cast<const char*>(p.in) + row[u] * p.row_bytes, at,
                  ok ? clamp8(p.H - at) : 0, p.vec != 0, raw[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t most = mx_largest<XD>(raw[u]);
    uint32_t o = from_lane<kQuadXor1>(most);
    most = o > most ? o : most;
    o = from_lane<kQuadXor2>(most);
    most = o > most ? o : most;
    const uint32_t scale = mx_scale(most);
    const uint32_t codes = mx_codes8<XD>(raw[u], scale);
    uint32_t word = scale << (8 * (lane >> 2));
    word |= from_lane<kRowRor4>(word);
    word |= from_lane<kRowRor8>(word);
    if (first_item() + u * 4 < p.items) {
      char* c = static_cast<char*>(p.codes) + row[u] * p.code_stride;
      *reinterpret_cast<uint32_t*>(c + (int64_t)g[u] * 64 + lane * 4) = codes;
      if (lane == 0)
        *reinterpret_cast<uint32_t*>(static_cast<char*>(p.scales) + row[u] * p.scale_stride +
                                     (int64_t)g[u] * 4) = word;
    }
  }
}

template <int OD>
__global__ __launch_bounds__(kMxThreads) void mx_dequantize(MxParams p) {
  constexpr int U = kMxUnroll;
  const int lane = threadIdx.x & 15;
  uint32_t row[U], g[U], codes[U], word[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t item = first_item() + u * 4;
    const bool ok = item < p.items;
    row[u] = ok ? limits::divide(item, p.by_groups) : 0;
    g[u] = item - row[u] * p.groups;
    int64_t src = ok ? row[u] : -1;
    if (ok && p.rows) src = p.rows[row[u]];
    codes[u] = word[u] = 0;  // a row that there is not: zeros
    if (src >= 0 && src < p.R) {
      codes[u] = *reinterpret_cast<const uint32_t*>(static_cast<const char*>(p.codes) +
                                                    src * p.code_stride + (int64_t)g[u] * 64 + lane * 4);
      word[u] = *reinterpret_cast<const uint32_t*>(static_cast<const char*>(p.scales) +
                                                   src * p.scale_stride + (int64_t)g[u] * 4);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (first_item() + u * 4 >= p.items) continue;
    u32x4 raw[raw_vecs<OD>()];
    mx_values8<OD>(codes[u], word[u] >> (8 * (lane >> 2)) & 255u, raw);
    const int64_t at = (int64_t)g[u] * 128 + lane * 8;
    char* out = static_cast<char*>(p.out) + row[u] * p.row_bytes;
    const int cnt = clamp8(p.H - at);
    if (p.vec && cnt == 8) {
      store_vec8<OD>(out, at, raw);
    } else {
      for (int i = 0; i < cnt; ++i) {
        if constexpr (OD == F32)
          reinterpret_cast<uint32_t*>(out)[at + i] = raw[i / 4][i % 4];
        else
          reinterpret_cast<uint16_t*>(out)[at + i] = (uint16_t)(raw[0][i / 2] >> (16 * (i % 2)));
      }
    }
  }
}

}  // namespace dev

const void* mx_quantize_kernel(int xd) {
  using namespace dev;
  return xd == F16 ? (const void*)mx_quantize<F16>
         : xd == BF16 ? (const void*)mx_quantize<BF16>
                      : (const void*)mx_quantize<F32>;
}

const void* mx_dequantize_kernel(int od) {
  using namespace dev;
  return od == F16 ? (const void*)mx_dequantize<F16>
         : od == BF16 ? (const void*)mx_dequantize<BF16>
                      : (const void*)mx_dequantize<F32>;
}

}  // namespace sgmv
