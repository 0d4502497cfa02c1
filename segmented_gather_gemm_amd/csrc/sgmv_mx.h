// sgmv_mx.h -- gfx950 device helpers of microscaled 4-bit values: blocks of 32
// consecutive values of a row that share a power of two.  Internal to libsgmv.
//
// A code is a sign (bit 3) and one of 0, .5, 1, 1.5, 2, 3, 4, 6; a block's
// scale byte s stands for 2^(s - 127), 255 for NaN.  The scale of a block whose
// largest magnitude is m is 2^(floor(log2 m) - 2), so that m lies in [4, 8) of
// it, and values above 6 become 6.  The conversion instructions round to the
// nearest value, ties to the even code, for every 16-bit value and scale, and
// read a scale's exponent bits alone, 0 as 2^-127 (all checked on the device).
#pragma once

#include <type_traits>

#include "sgmv_common.h"

namespace sgmv {
namespace dev {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// D = A . B + C on 16 x 16 float32, A 16 x 128 and B 128 x 16 of 4-bit values:
// lane l holds block l / 16 of row (column) l % 16, and byte SEL of `sa` and
// `sb` its scale.  Products are exact; a NaN scale makes the products NaN.
template <int SEL>
__device__ __forceinline__ f32x4 mfma_fp4(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, SEL, (int)sa, SEL,
                                                          (int)sb);
}

// The scale byte of a block whose largest magnitude has these float32 bits
// (magnitudes below 2^-126 end at 2^-127 as zero does; infinity and NaN: 255).
__device__ __forceinline__ uint32_t mx_scale(uint32_t largest) {
  const uint32_t e = largest >> 23;
  return e == 255 ? 255 : e < 2 ? 0 : e - 2;
}

// Bits of the largest magnitude, as float32, of values in packed words (16-bit:
// two a word).
template <int XD, int N>
__device__ __forceinline__ uint32_t mx_largest(const u32x4 (&raw)[N]) {
  if constexpr (XD == F32) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t m = raw[i][j] & 0x7FFFFFFFu;
        most = m > most ? m : most;
      }
    return most;
  } else {
    u16x2 most = {0, 0};
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        most = __builtin_elementwise_max(
            most, __builtin_bit_cast(u16x2, (uint32_t)(raw[i][j] & 0x7FFF7FFFu)));
    const uint32_t m = most.x > most.y ? most.x : most.y;
    return __float_as_uint(widen<XD>(m));
  }
}

// Eight values (one 16-byte block, two of float32) as eight codes.
template <int XD>
__device__ __forceinline__ uint32_t mx_codes8(const u32x4* raw, uint32_t scale) {
  const float s = __uint_as_float(scale << 23);
  uint32_t c = 0;
  if constexpr (XD == BF16) {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)raw[0][0]), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)raw[0][1]), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)raw[0][2]), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)raw[0][3]), s, 3);
  } else if constexpr (XD == F16) {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, (uint32_t)raw[0][0]), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, (uint32_t)raw[0][1]), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, (uint32_t)raw[0][2]), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(f16x2, (uint32_t)raw[0][3]), s, 3);
  } else {
    auto f = [&](int i) { return __uint_as_float(raw[i / 4][i % 4]); };
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f(0), f(1), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f(2), f(3), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f(4), f(5), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f(6), f(7), s, 3);
  }
  return scale == 255 ? 0 : c;
}

// Eight codes as the values of dtype OD they stand for (rounded where OD cannot
// hold them: float16's ends, and past float32's largest).
template <int OD>
__device__ __forceinline__ void mx_values8(uint32_t codes, uint32_t scale, u32x4* raw) {
  const float s = __uint_as_float(scale == 0 ? 0x00400000u : scale << 23);
  auto put = [&](auto sel) {
    constexpr int i = decltype(sel)::value;
    if constexpr (OD == F32) {
      const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, i);
      raw[i / 2][2 * (i % 2)] = __float_as_uint(v.x);
      raw[i / 2][2 * (i % 2) + 1] = __float_as_uint(v.y);
    } else if constexpr (OD == BF16) {
      raw[0][i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, i));
    } else {
      raw[0][i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, s, i));
    }
  };
  put(std::integral_constant<int, 0>{});
  put(std::integral_constant<int, 1>{});
  put(std::integral_constant<int, 2>{});
  put(std::integral_constant<int, 3>{});
  if (scale == 255) {
    constexpr uint32_t kNan = OD == F32 ? 0x7FC00000u : OD == BF16 ? 0x7FC07FC0u : 0x7E007E00u;
#pragma unroll
    for (int i = 0; i < raw_vecs<OD>(); ++i) raw[i] = u32x4{kNan, kNan, kNan, kNan};
  }
}

// The sum of a value over the wave, in all lanes.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

}  // namespace dev
}  // namespace sgmv
