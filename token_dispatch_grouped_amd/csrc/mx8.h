// The 8-bit block form (MOE_DTYPE_MX8) on the device: e4m3 elements and one
// power-of-two scale (an e8m0 byte, 2^(code - 127)) for each 32 consecutive
// elements of a row.
#pragma once

#include "common.h"

namespace moe {

constexpr int kMx8Block = 32;

// Scale code of a block whose largest |value| has the fp32 pattern
// `amax_bits`: the smallest power of two S with amax <= 448 S. With amax =
// 1.f * 2^E and 448 = 1.75 * 2^8, S = 2^(E-8), or 2^(E-7) once 1.f > 1.75:
// exact integer arithmetic, so no rounding decides a scale. Blocks below
// 448 * 2^-127 (zero among them) take code 0; a block that holds an infinity
// or a NaN takes 255, the scale that is no number.
MOE_DEVICE uint32_t mx8_scale_code(uint32_t amax_bits) {
  const int c = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return amax_bits >= 0x7f800000u ? 255u : (uint32_t)(c < 0 ? 0 : c);
}

// 1 / S = 2^(127 - code): codes 0 .. 247 give normal fp32 numbers. Code 255
// gives NaN, so that every element of such a block is stored as NaN.
MOE_DEVICE float mx8_inv_scale(uint32_t code) {
  return code == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float((254u - code) << 23);
}

// Four scaled values to four e4m3 bytes, nearest-even (|v| <= 448 by the
// choice of the scale, so nothing saturates).
MOE_DEVICE uint32_t mx8_pack4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return (uint32_t)w;
}

MOE_DEVICE uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
MOE_DEVICE uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Cross-lane steps without LDS (DPP): the value of lane ^ 1, of lane ^ 2,
// of the mirrored lane within 8, and within 16.
template <int CTRL>
MOE_DEVICE uint32_t dpp_u(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xf, 0xf, false);
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppMirror8 = 0x141, kDppMirror16 = 0x140;

// Maximum over groups of N consecutive lanes (N = 4 or 8), in every lane.
template <int N>
MOE_DEVICE uint32_t group_umax(uint32_t v) {
  static_assert(N == 4 || N == 8, "a block is four lanes of 8 elements or eight of 4");
  v = umax(v, dpp_u<kDppXor1>(v));
  v = umax(v, dpp_u<kDppXor2>(v));
  if (N == 8) v = umax(v, dpp_u<kDppMirror8>(v));
  return v;
}

// Sum over a wavefront, the same bits in every lane: DPP within 16 lanes,
// two LDS-crossbar steps beyond.
MOE_DEVICE float wave_sum_dpp(float v) {
  v += __uint_as_float(dpp_u<kDppXor1>(__float_as_uint(v)));
  v += __uint_as_float(dpp_u<kDppXor2>(__float_as_uint(v)));
  v += __uint_as_float(dpp_u<kDppMirror8>(__float_as_uint(v)));
  v += __uint_as_float(dpp_u<kDppMirror16>(__float_as_uint(v)));
  v += __shfl_xor(v, 16, kWave);
  v += __shfl_xor(v, 32, kWave);
  return v;
}

}  // namespace moe
