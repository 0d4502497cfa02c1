// Kernels that quantise rows to microscaled 4-bit values and read them back.
//
// A lane has eight values (16 bytes of 16-bit ones), four lanes a block of 32,
// sixteen lanes a group of 128: the block's largest magnitude takes two
// exchanges inside a quad of lanes, loads and stores are consecutive over the
// lanes, and a group's four scale bytes leave as one word.  Groups are dealt to
// the lanes over all rows, whatever a row's length.  Bound by memory: 16384 x
// 4096 bfloat16 values 31.0 us = 5.5 TB/s, 28672 x 4096 float32 ones 110 us = 4.8
// TB/s and back to bfloat16 55 us = 5.4 TB/s (a copy of 1 GiB 5.1); kMxUnroll
// groups a lane, two against one, four and eight: 31.0, 32.6, 31.9 and 33.0 us.
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

// A block of eight values as its codes, and its block's scale byte (of the four
// lanes that hold a block of 32; all lanes take part).
template <int XD>
__device__ __forceinline__ uint32_t quantize8(const u32x4 (&raw)[raw_vecs<XD>()], uint32_t* scale) {
  uint32_t most = mx_largest<XD>(raw);
  uint32_t o = from_lane<kQuadXor1>(most);
  most = o > most ? o : most;
  o = from_lane<kQuadXor2>(most);
  most = o > most ? o : most;
  *scale = mx_scale(most);
  return mx_codes8<XD>(raw, *scale);
}

// The scale bytes of a group's four blocks as one word (in all sixteen lanes).
__device__ __forceinline__ uint32_t scale_word(uint32_t scale) {
  uint32_t word = scale << (8 * ((threadIdx.x & 15) >> 2));
  word |= from_lane<kRowRor4>(word);
  return word | from_lane<kRowRor8>(word);
}

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
    uint32_t scale;
    const uint32_t codes = quantize8<XD>(raw[u], &scale);
    const uint32_t word = scale_word(scale);
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

// One token and eight rows of its adapter's lora_A for a slice: a wave has one of
// the rows and the token's values, eight a lane and 512 at a time, so that all
// of a row's loads are in flight together.  Bound by their latency: a decode
// batch of 64 tokens, 32 adapters and three slices of rank 16 (hidden 4096) takes
// 7.2-7.6 us (two rows a wave 8.4); the kernels it replaces, which gather each
// adapter's tokens for the matrix unit, 3.7 and 11.
template <int XD>
__global__ __launch_bounds__(64 * kMxProjectWaves) void mx_project(MxProjectParams p) {
  constexpr int kAhead = kMxProjectAhead;
  __shared__ int32_t adapter;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int part = blockIdx.x % p.parts, slice = blockIdx.x / p.parts, t = blockIdx.y;
  const char* x = static_cast<const char*>(p.x) + t * p.x_row_bytes;
  const int groups = (p.H + 127) / 128;
  u32x4 xv[kAhead][1];
  auto read_x = [&](int base) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int at = (base + i * 64 + lane) * 8;
      xv[i][0] = u32x4{};
      if (at < p.H) xv[i][0] = *reinterpret_cast<const u32x4*>(x + (int64_t)at * 2);
    }
  };
  read_x(0);  // ahead of the search for the token's adapter
  if (threadIdx.x == 0) adapter = -1;
  __syncthreads();
  for (int32_t b = threadIdx.x; b < p.batches; b += 64 * kMxProjectWaves) {
    const int64_t st = p.start[b], ln = p.lens[b], a = p.idx[b];
    if (a >= 0 && a < p.L && ln > 0 && st >= 0 && st <= p.T - ln && st <= t && t < st + ln)
      adapter = (int32_t)a;  // segments are disjoint
  }
  const bool quantise = p.codes != nullptr && blockIdx.x == 0;
  __syncthreads();
  const int a = uniform(adapter);
  if (a < 0 && !quantise) return;
  const int k0 = part * kMxProjectRows + wave;
  const bool have = a >= 0 && k0 < p.K;
  // p.a and p.v by a variable index would be copied to scratch memory.
  typedef const __attribute__((address_space(4))) MxProjectParams* Args;
  const Args args = (Args)__builtin_amdgcn_kernarg_segment_ptr();
  const int64_t row_bytes = (int64_t)p.H * 2;
  const char* la = static_cast<const char*>(args->a[slice]) + ((int64_t)(a < 0 ? 0 : a) * p.K + k0) * row_bytes;
  float sum = 0.f;
  for (int base = 0; base < groups * 16; base += 64 * kAhead) {
    u32x4 av[kAhead];
    if (base > 0) read_x(base);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int at = (base + i * 64 + lane) * 8;
      av[i] = u32x4{};
      if (at < p.H && have) av[i] = *reinterpret_cast<const u32x4*>(la + (int64_t)at * 2);
    }
    // A wave quantises one block a lane, whole groups of the row.
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (!quantise || i != wave) continue;
      uint32_t scale;
      const uint32_t codes = quantize8<XD>(xv[i], &scale);
      const uint32_t word = scale_word(scale);
      const int g = (base + i * 64 + lane) / 16;
      if (g < groups) {
        char* c = static_cast<char*>(p.codes) + t * p.code_stride;
        reinterpret_cast<uint32_t*>(c)[base + i * 64 + lane] = codes;
        if ((lane & 15) == 0)
          reinterpret_cast<uint32_t*>(static_cast<char*>(p.scales) + t * p.scale_stride)[g] = word;
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      float xf[8], f[8];
      out_values<XD>(xv[i], xf);
      out_values<XD>(&av[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(xf[j], f[j], sum);
    }
  }
  sum = wave_sum(sum) * p.scale;
  if (lane == 0 && have) args->v[slice][(int64_t)t * p.v_stride + k0] = sum;
}

}  // namespace dev

const void* mx_project_kernel(int xd) {
  using namespace dev;
  static_assert(kMxProjectWaves == 8, "a wave quantises one of its eight blocks a lane");
  return xd == BF16 ? (const void*)mx_project<BF16> : (const void*)mx_project<F16>;
}

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
