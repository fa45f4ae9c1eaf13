// out = A B^T of 8-bit matrices with a power of two as the scale of each 128 values along K.
//
// The matrix instruction 16x16x128 takes 8-bit operands with a scale for each 32 values of a
// row, so one instruction is a group's product with its scales applied, and nothing is
// left for the vector units.  Inside, products are summed with fewer bits than fp32 has
// (measured: off by 1.5e-5 of the result's norm for normal values, 7e-5 where they span eight
// powers of two), which outputs of 16 bits do not show; a float32 output is taken
// by the bf16 instruction, whose products are exact and whose sums are fp32, after the 8 bits
// and their scales are turned into bf16 (exact), at about half the rate.
//
// The product is taken transposed (B's rows as the instruction's rows), so that a lane holds
// four neighbouring columns of a row of out.
#include "fp8.h"
#include "fp8_device.h"
#include "vec.h"

namespace s4 {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr int kK = 128;   // values along K a step: one group

// What lies behind a matrix's last column.
__device__ __attribute__((aligned(16))) const unsigned kZeros[4] = {0, 0, 0, 0};

// The scales of groups kb .. kb + 3 of a row, byte 0 the first (behind the row's end anything).
__device__ __forceinline__ unsigned scales4(const unsigned char* __restrict__ row, int kb, int n) {
  if (n >= 4) {   // the same for all lanes
    const int at = kb < n - 4 ? kb : n - 4;
    unsigned t;
    __builtin_memcpy(&t, row + at, 4);
    return t >> (8 * (kb - at));
  }
  unsigned t = 0;
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (kb + i < n) t |= (unsigned)row[kb + i] << (8 * i);
  return t;
}

__device__ __forceinline__ float scale_value(unsigned byte) {   // 2^(byte - 127), NaN for 255
  return byte == 255 ? __uint_as_float(0x7fc00000u)
                     : byte ? __uint_as_float(byte << 23) : __uint_as_float(0x00400000u);
}

// 32 e4m3 values times a scale as four operands of the bf16 instruction.
__device__ __forceinline__ void widen(v8i x, float scale, v8bf (&out)[4]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const v2bf lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)x[i], scale, false);
    const v2bf hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)x[i], scale, true);
    out[i / 2][4 * (i % 2)] = lo[0];
    out[i / 2][4 * (i % 2) + 1] = lo[1];
    out[i / 2][4 * (i % 2) + 2] = hi[0];
    out[i / 2][4 * (i % 2) + 3] = hi[1];
  }
}

// Columns n .. n + 3 of row m of out.
template <typename T>
__device__ __forceinline__ void store4(T* __restrict__ out, long ldo, int m, int n, int M, int N,
                                       v4f c) {
  if (m >= M) return;
  T* p = out + (long)m * ldo + n;
  T t[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) t[e] = from_f32<T>(c[e]);
  if (n + 4 <= N) {
    __builtin_memcpy(p, t, sizeof(t));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < N) p[e] = t[e];
  }
}

// Block -> tile.  Blocks go round robin over the 8 XCDs, so each XCD takes a run of neighbouring
// tiles; a run goes down 8 tiles of M before the next tile of N, which keeps its operands in the
// XCD's own L2.
__device__ __forceinline__ bool tile_of(int mt, int nt, int* m, int* n) {
  const long total = (long)mt * nt;
  const unsigned per = gridDim.x / 8, id = blockIdx.x % 8 * per + blockIdx.x / 8;
  if (id >= total) return false;
  const unsigned band = id / (8u * nt), in = id % (8u * nt);
  const unsigned left = mt - band * 8, rows = left < 8 ? left : 8;
  *m = band * 8 + in % rows;
  *n = in / rows;
  return true;
}

}  // namespace

// A block takes BM x BN of out, a wave WM x WN of it.  Both operands' next step is on its way
// to the other half of LDS while one is computed: 128 rows of 128 bytes, 16-byte piece p of row
// r at p ^ (r / 2 % 8), so that the 16 rows of an operand's read lie in different banks.
// WHOLE: rows start at multiples of 16 bytes and K is one, so that pieces are whole and go to LDS
// without registers.
template <typename T, int BM, int BN, int WM, int WN, bool WHOLE>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) void matmul_kernel(const MatmulArgs p) {
  constexpr bool kExact = sizeof(T) == 4;
  constexpr int WAVES = (BM / WM) * (BN / WN), MT = WM / 16, NT = WN / 16;
  constexpr int LOADS = (BM + BN) / 8;   // of 8 rows, 16 bytes a lane
  __shared__ __attribute__((aligned(16))) unsigned char lds[2][(BM + BN) * kK];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int m0, n0;
  if (!tile_of((p.M + BM - 1) / BM, (p.N + BN - 1) / BN, &m0, &n0)) return;
  m0 *= BM;
  n0 *= BN;
  const int wm = w / (BN / WN) * WM, wn = w % (BN / WN) * WN;
  const int steps = (p.K + kK - 1) / kK;

  auto stage = [&](int kb, int buf) {
#pragma unroll
    for (int i = 0; i < (LOADS + WAVES - 1) / WAVES; ++i) {
      const int at = i * WAVES + w;
      if (LOADS % WAVES && at >= LOADS) break;
      const int r = at * 8 + lane / 8, piece = (lane % 8) ^ (r / 2 % 8);
      const bool left = at < BM / 8;
      const int most = (left ? p.M : p.N) - 1;
      int row = left ? m0 + r : n0 + r - BM;
      row = row < most ? row : most;   // rows behind the end: the last one, not stored
      const unsigned char* src = left ? p.a + (long)row * p.lda : p.b + (long)row * p.ldb;
      const int k = kb * kK + piece * 16;
      if constexpr (WHOLE) {
        src = k < p.K ? src + k : reinterpret_cast<const unsigned char*>(kZeros);
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) void*)src,
            (__attribute__((address_space(3))) void*)&lds[buf][at * 1024], 16, 0, 0);
      } else {
        unsigned char t[16];
        if (k + 16 <= p.K) {
          __builtin_memcpy(t, src + k, 16);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) t[j] = k + j < p.K ? src[k + j] : 0;
        }
        __builtin_memcpy(&lds[buf][at * 1024 + lane * 16], t, 16);
      }
    }
  };
  auto operand = [&](int buf, int row) {   // row: a multiple of 16
    const int r = lane & 15, g = lane >> 4;
    const unsigned char* at = &lds[buf][(row + r) * kK];
    v8i x;
    __builtin_memcpy(&x, at + ((2 * g) ^ (r / 2)) * 16, 16);
    __builtin_memcpy((char*)&x + 16, at + ((2 * g + 1) ^ (r / 2)) * 16, 16);
    return x;
  };

  v4f acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  // rows of the scales that this lane's rows have
  const unsigned char *sa[MT], *sb[NT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = m0 + wm + 16 * i + (lane & 15);
    sa[i] = p.sa + (long)(m < p.M ? m : p.M - 1) * steps;
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    int n = n0 + wn + 16 * j + (lane & 15);
    n = n < p.N ? n : p.N - 1;
    sb[j] = p.sb + (long)(p.square ? n / kGroup : n) * steps;
  }
  unsigned ea[MT], eb[NT];
  if (steps > 0) stage(0, 0);
  for (int kb = 0; kb < steps; ++kb) {
    if (kb % 4 == 0) {
#pragma unroll
      for (int i = 0; i < MT; ++i) ea[i] = scales4(sa[i], kb, steps);
#pragma unroll
      for (int j = 0; j < NT; ++j) eb[j] = scales4(sb[j], kb, steps);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (kb + 1 < steps) stage(kb + 1, (kb + 1) & 1);
    const int buf = kb & 1;
    if constexpr (kExact) {
      v8bf a[MT][4];
#pragma unroll
      for (int i = 0; i < MT; ++i) widen(operand(buf, wm + 16 * i), scale_value(ea[i] & 255), a[i]);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        v8bf b[4];
        widen(operand(buf, BM + wn + 16 * j), scale_value(eb[j] & 255), b);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[q], a[i][q], acc[i][j], 0, 0, 0);
      }
    } else {
      v8i a[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) a[i] = operand(buf, wm + 16 * i);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const v8i b = operand(buf, BM + wn + 16 * j);
#pragma unroll
        for (int i = 0; i < MT; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              b, a[i], acc[i][j], 0, 0, 0, (int)eb[j], 0, (int)ea[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) ea[i] >>= 8;
#pragma unroll
    for (int j = 0; j < NT; ++j) eb[j] >>= 8;
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
      store4((T*)p.out, p.ldo, m0 + wm + 16 * i + (lane & 15), n0 + wn + 16 * j + 4 * (lane >> 4),
             p.M, p.N, acc[i][j]);
}

namespace {

template <typename T, int BM, int BN, int WM, int WN>
hipError_t tiles(const MatmulArgs& a, bool whole, hipStream_t s) {
  const long n = (long)((a.N + BN - 1) / BN) * ((a.M + BM - 1) / BM);
  const unsigned grid = (unsigned)((n + 7) / 8 * 8);
  constexpr int threads = (BM / WM) * (BN / WN) * 64;
  if (whole) matmul_kernel<T, BM, BN, WM, WN, true><<<grid, threads, 0, s>>>(a);
  else matmul_kernel<T, BM, BN, WM, WN, false><<<grid, threads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t matmul(const MatmulArgs& a, hipStream_t s) {
  const bool whole = ((reinterpret_cast<uintptr_t>(a.a) | reinterpret_cast<uintptr_t>(a.b) |
                       (uintptr_t)a.lda | (uintptr_t)a.ldb | (uintptr_t)a.K) & 15) == 0;
  return tiles<T, 128, 128, 64, 64>(a, whole, s);
}

}  // namespace

hipError_t launch_matmul(const MatmulArgs& a, int dtype, hipStream_t s) {
  if (dtype == S4DPLR_F32) return matmul<float>(a, s);
  return dtype == S4DPLR_BF16 ? matmul<bf16>(a, s) : matmul<f16>(a, s);
}

}  // namespace s4
