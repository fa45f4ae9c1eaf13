// 8-bit floating point with a power of two as the scale of a group of 128: e4m3 values
// (largest 448) and e8m0 scales (byte b stands for 2^(b - 127), 255 for NaN).
#pragma once

#include "vec.h"

namespace s4 {

constexpr int kGroup = 128;   // values that share a scale

// The larger of two values by the bits of their magnitudes, which order NaN above infinity.
__device__ __forceinline__ unsigned magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }
template <int CTRL>
__device__ __forceinline__ unsigned max_dpp(unsigned v) {
  const unsigned o = (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
  return o > v ? o : v;
}
// Largest over every N = 16 or 32 neighbouring lanes, in all of them.
template <int N>
__device__ __forceinline__ unsigned max_of(unsigned v) {
  static_assert(N == 16 || N == 32, "");
  v = max_dpp<0xB1>(v);    // quad_perm [1, 0, 3, 2]
  v = max_dpp<0x4E>(v);    // quad_perm [2, 3, 0, 1]
  v = max_dpp<0x141>(v);   // row_half_mirror
  v = max_dpp<0x140>(v);   // row_mirror
  if constexpr (N == 32) {
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = a[0] > a[1] ? a[0] : a[1];
  }
  return v;
}

// The scale of a group whose largest magnitude has these bits: the least power of two s with
// magnitude <= 448 s, 2^-126 at least; NaN for an infinity or NaN.  A value times a power
// of two is exact, so the one rounding of quantization is that to e4m3, and a
// product's scales cost its sums nothing (with a scale of magnitude / 448 they would).
__device__ __forceinline__ unsigned scale_byte(unsigned bits) {
  if (bits >= 0x7f800000u) return 255;
  // 448 = 1.75 2^8
  const int e = (int)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return (unsigned)(e > 1 ? e : 1);
}
__device__ __forceinline__ float inverse_scale(unsigned byte) {   // NaN stays NaN
  return byte == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float((254 - byte) << 23);
}

// Four values, of magnitude 448 or less, to e4m3 (nearest, ties to even).
__device__ __forceinline__ unsigned pack4(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

}  // namespace s4
