// Element types and small helpers shared by the token-major operators.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

namespace s4 {

typedef __bf16 bf16;
typedef _Float16 f16;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16 v) { return (float)v; }
__device__ __forceinline__ float to_f32(f16 v) { return (float)v; }
// one rounding to nearest even at every store
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  return (T)v;
}

// 16 bytes of elements; the source needs no more than the element's own
// alignment (the compiler emits one 16-byte load: global memory takes any
// address on this target).
template <typename T>
struct Vec {
  static constexpr int N = 16 / (int)sizeof(T);
  T v[N];
};

template <typename T>
__device__ __forceinline__ Vec<T> load_vec(const T* p) {
  Vec<T> r;
  __builtin_memcpy(&r, p, sizeof(r));
  return r;
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const Vec<T>& r) {
  __builtin_memcpy(p, &r, sizeof(r));
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}

// Sum over each row of 16 lanes, in every lane: lanes xor 1, xor 2, then the
// mirrored halves and the mirrored row (whose partners hold equal sums).
__device__ __forceinline__ float sum16(float v) {
  v += dpp<0xB1>(v);    // quad_perm [1, 0, 3, 2]
  v += dpp<0x4E>(v);    // quad_perm [2, 3, 0, 1]
  v += dpp<0x141>(v);   // row_half_mirror
  v += dpp<0x140>(v);   // row_mirror
  return v;
}

// Sum over the 64 lanes, in every lane: rows 0 + 1 and 2 + 3, then the halves (the
// swaps hand over the other row or half).
__device__ __forceinline__ float sum64(float v) {
  v = sum16(v);
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

}  // namespace s4
