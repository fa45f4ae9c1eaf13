// Rows of D contiguous values held by the waves of a block: what the norms over rows share.
#pragma once

#include "vec.h"

namespace s4 {

constexpr int kRowThreads = 256;

// A lane's share of a row as it lies in memory: NV vectors, vector i at element
// ((i WPR + wave) 64 + lane) VEC.  WHOLE: D is a multiple of VEC, so a vector is
// inside or outside; one outside is read from the row's start and replaced by 0, with
// no branch for the loads to wait at.
template <typename T, int NV, int WPR, bool WHOLE>
struct RowPart {
  static constexpr int VEC = Vec<T>::N, E = NV * VEC;
  Vec<T> v[NV];
  __device__ __forceinline__ static int at(int i, int tid) { return (i * WPR * 64 + tid) * VEC; }
  __device__ __forceinline__ void load(const T* __restrict__ p, int D, int tid) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = at(i, tid);
      if constexpr (WHOLE) {
        v[i] = load_vec(p + (c < D ? c : 0));
      } else if (c + VEC <= D) {
        v[i] = load_vec(p + c);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i].v[j] = c + j < D ? p[c + j] : (T)0.f;
      }
    }
  }
  __device__ __forceinline__ void get(int D, int tid, float* out) const {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        out[i * VEC + j] = !WHOLE || at(i, tid) < D ? to_f32(v[i].v[j]) : 0.f;
  }
  __device__ __forceinline__ static void store(T* __restrict__ p, int D, int tid, const float* in) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = at(i, tid);
      if (c + VEC <= D) {
        Vec<T> t;
#pragma unroll
        for (int j = 0; j < VEC; ++j) t.v[j] = from_f32<T>(in[i * VEC + j]);
        store_vec(p + c, t);
      } else if constexpr (!WHOLE) {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (c + j < D) p[c + j] = from_f32<T>(in[i * VEC + j]);
      }
    }
  }
  // the same columns of a vector of D floats; `other` where there is none
  __device__ __forceinline__ static void columns(const float* __restrict__ p, int D, int tid,
                                                 float other, float* out) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = at(i, tid);
      if (p && c + VEC <= D) {
        __builtin_memcpy(out + i * VEC, p + c, VEC * sizeof(float));
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) out[i * VEC + j] = p && c + j < D ? p[c + j] : other;
      }
    }
  }
};

// Rows of 32 values a lane over 16 waves: those have 128 registers a lane, so gamma and beta
// are read where they are used (2048 x 32768 bf16 108 -> 72 us; 60 since the forward pass joins
// its waves' parts a lane each, which leaves it without spills; fp32 114).
constexpr bool wide_rows(int values, int waves) { return waves > 4 && values > 16; }

// The same value, unknown to the compiler: a load at it is not taken out of the loop, where
// its result would be kept in registers and spilled.
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Sum over every group of N lanes, 4 or 16, the same bits in all of them: a lane's own product
// must not enter the first addition unrounded, as a contraction would have it.
template <int N>
__device__ __forceinline__ float sum_of(float v) {
#pragma clang fp contract(off)
  static_assert(N == 4 || N == 16, "");
  v += dpp<0xB1>(v);    // quad_perm [1, 0, 3, 2]
  v += dpp<0x4E>(v);    // quad_perm [2, 3, 0, 1]
  if constexpr (N == 16) {
    v += dpp<0x141>(v);   // row_half_mirror
    v += dpp<0x140>(v);   // row_mirror
  }
  return v;
}

// Both sums over the waves of a row, in every lane; `red` is used in turn.
template <int WPR>
__device__ __forceinline__ void block_sums(float& s1, float& s2, float (&red)[2][WPR]) {
  s1 = sum64(s1);
  s2 = sum64(s2);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) {
      red[0][threadIdx.x >> 6] = s1;
      red[1][threadIdx.x >> 6] = s2;
    }
    __syncthreads();
    s1 = s2 = 0.f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) {
      s1 += red[0][i];
      s2 += red[1][i];
    }
  }
}

inline long ceil_div(long a, long b) { return (a + b - 1) / b; }

// Vectors a lane holds and waves a row takes: one wave up to 2 vectors a lane, then
// 4 waves, then 16.  On either side: one wave with 4 vectors, 16384 x 2048 bf16 backward
// 41.1 us instead of 38.8 (forward 23.3 instead of 28.7); 4 waves from 2 vectors on, 65536 x
// 512 fp32 forward 76.6 us instead of 45.8, backward 124 instead of 75; 16 waves from 16
// vectors on, 8192 x 8192 bf16 forward 55.5 us instead of 43.6, backward 80.5 instead of 81.9.
template <typename T, typename F>
void row_shape(int D, F f) {
  const int vecs = (int)ceil_div(D, 64 * Vec<T>::N);
  const bool whole = D % Vec<T>::N == 0;
  using std::integral_constant;
  using Yes = std::true_type;
  using No = std::false_type;
#define S4_CASE(nv, wpr)                                                                 \
  (whole ? f(integral_constant<int, nv>(), integral_constant<int, wpr>(), Yes())         \
         : f(integral_constant<int, nv>(), integral_constant<int, wpr>(), No()))
  if (vecs <= 1) return S4_CASE(1, 1);
  if (vecs <= 2) return S4_CASE(2, 1);
  if (vecs <= 4) return S4_CASE(1, 4);
  if (vecs <= 8) return S4_CASE(2, 4);
  if (vecs <= 16) return S4_CASE(4, 4);
  if (vecs <= 32) return S4_CASE(2, 16);
  if (vecs <= 64) return S4_CASE(4, 16);
  if constexpr (sizeof(T) == 4) return S4_CASE(8, 16);
#undef S4_CASE
}

}  // namespace s4
