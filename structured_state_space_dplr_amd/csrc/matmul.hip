// out = A B^T of 8-bit matrices with a power of two as the scale of each 128 values along K.
//
// The matrix instruction 16x16x128 takes 8-bit operands with a scale for each 32 values of a
// row, so one instruction is a group's product with its scales applied, and nothing is
// left for the vector units.  Inside, products are summed with fewer bits than fp32 has
// (measured: off by 1.5e-5 of the result's norm for normal values, 7e-5 where both operands' span
// eight powers of two, up to about 2^-13 of a group's sum of magnitudes), which outputs of 16 bits
// rarely show; a float32 output is taken by the bf16 instruction, whose products are exact and
// whose sums are fp32, after the 8 bits and their scales are turned into bf16 (exact), at about half
// the rate (4096^3: 1.8 PFLOP/s in bf16, 1.0 in float32).
//
// The product is taken transposed (B's rows as the instruction's rows), so that a lane holds
// four neighbouring columns of a row of out.
#include "fp8.h"
#include "fp8_device.h"
#include "vec.h"

namespace s4 {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr int kK = 128;   // values along K a step: one group

// What lies behind a matrix's last column.
__device__ __attribute__((aligned(16))) const unsigned kZeros[4] = {0, 0, 0, 0};

// The scales of groups kb .. kb + 3 of R rows (behind a row's end anything): byte 0 is the first once
// they are shifted by scales_shift, which waits for the loads.
__device__ __forceinline__ int scales_shift(int kb, int n) {
  return n >= 4 && kb > n - 4 ? 8 * (kb - (n - 4)) : 0;
}
template <int R>
__device__ __forceinline__ void scales4(const unsigned char* const (&row)[R], int kb, int n,
                                        unsigned (&out)[R]) {
  if (n >= 4) {   // the same for all lanes, and no load under another condition
    const int at = kb < n - 4 ? kb : n - 4;
#pragma unroll
    for (int i = 0; i < R; ++i) __builtin_memcpy(&out[i], row[i] + at, 4);
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      out[i] = 0;
      for (int j = 0; kb + j < n; ++j) out[i] |= (unsigned)row[i][kb + j] << (8 * j);
    }
  }
}

// Bytes k .. k + 16 of a row of K, as they lie 16 bytes before its end where it ends sooner: one load,
// not one a byte.  piece_end moves them to their place, with zeros behind the end.
__device__ __forceinline__ v4i piece16(const unsigned char* __restrict__ row, int k, int K) {
  v4i x = {0, 0, 0, 0};
  if (K >= 16) {   // the same for all lanes
    __builtin_memcpy(&x, row + (k < K - 16 ? k : K - 16), 16);
  } else {
    unsigned long lo = 0, hi = 0;
    for (int j = 0; j < K; ++j) {
      const unsigned long v = row[j];
      if (j < 8) lo |= v << (8 * j);
      else hi |= v << (8 * (j - 8));
    }
    x = v4i{(int)lo, (int)(lo >> 32), (int)hi, (int)(hi >> 32)};
  }
  return x;
}
__device__ __forceinline__ v4i piece_end(v4i x, int k, int K) {
  const int cut = K >= 16 ? k - (k < K - 16 ? k : K - 16) : k;   // bytes before k
  unsigned long lo, hi;
  __builtin_memcpy(&lo, &x, 8);
  __builtin_memcpy(&hi, (const char*)&x + 8, 8);
  if (cut >= 16) {
    lo = hi = 0;
  } else if (cut >= 8) {
    lo = hi >> (8 * (cut - 8));
    hi = 0;
  } else {
    lo = lo >> (8 * cut) | (hi << 1) << (63 - 8 * cut);
    hi >>= 8 * cut;
  }
  return v4i{(int)lo, (int)(lo >> 32), (int)hi, (int)(hi >> 32)};
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

// The operand that a lane holds: 32 bytes of row lane % 16 behind byte 32 (lane / 16) of a group.
// c += b a for MT x NT tiles of 16 x 16, one group along K; sa, sb: the groups' scales in byte 0.
template <typename T, int MT, int NT, typename FA, typename FB>
__device__ __forceinline__ void group_product(FA a_of, FB b_of, const unsigned (&sa)[MT],
                                              const unsigned (&sb)[NT], v4f (&acc)[MT][NT]) {
  if constexpr (sizeof(T) == 4) {
    v8bf a[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i) widen(a_of(i), scale_value(sa[i] & 255), a[i]);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      v8bf b[4];
      widen(b_of(j), scale_value(sb[j] & 255), b);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < MT; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[q], a[i][q], acc[i][j], 0, 0, 0);
    }
  } else {
    v8i a[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) a[i] = a_of(i);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const v8i b = b_of(j);
#pragma unroll
      for (int i = 0; i < MT; ++i)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            b, a[i], acc[i][j], 0, 0, 0, (int)sb[j], 0, (int)sa[i]);
    }
  }
}

// A block takes BM x BN of out, a wave WM x WN of it.  Both operands' next step is on its way
// to the other half of LDS while one is computed: rows of 128 bytes, 16-byte piece p of row
// r at p ^ (r / 2 % 8), so that the 16 rows of an operand's read lie in different banks.  The
// halves are two variables and their steps written out in turn, without which the compiler waits
// for the loads before it reads the other half.
// WHOLE: rows start at multiples of 16 bytes and K is one, so that pieces are whole and go to LDS
// without registers.
// DEEP: three steps on their way to four buffers, for small tiles, whose steps are shorter than a load.
template <typename T, int BM, int BN, int WM, int WN, bool WHOLE, bool DEEP>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64, 2) void matmul_kernel(const MatmulArgs p) {
  constexpr int WAVES = (BM / WM) * (BN / WN), MT = WM / 16, NT = WN / 16;
  constexpr int LOADS = (BM + BN) / 8 / WAVES, LEFT = BM / 8 / WAVES;   // of 8 rows, 16 bytes a lane
  static_assert(LOADS * 8 * WAVES == BM + BN && LEFT * 8 * WAVES == BM, "");
  constexpr int BYTES = (BM + BN) * kK;
  __shared__ __attribute__((aligned(16))) unsigned char lds0[BYTES], lds1[BYTES],
      lds2[DEEP ? BYTES : 16], lds3[DEEP ? BYTES : 16];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int m0, n0;
  if (!tile_of((p.M + BM - 1) / BM, (p.N + BN - 1) / BN, &m0, &n0)) return;
  m0 *= BM;
  n0 *= BN;
  const int wm = w / (BN / WN) * WM, wn = w % (BN / WN) * WN;
  const int steps = (p.K + kK - 1) / kK;

  // rows of the block's loads as offsets of 32 bits (256 rows of less than 2^24 bytes)
  const unsigned char* const base_a = p.a + (long)m0 * p.lda;
  const unsigned char* const base_b = p.b + (long)n0 * p.ldb;
  unsigned from[LOADS];
  const int lrow = lane / 8;
  // 8 rows a load: those of a wave's loads are 8 WAVES apart, their turn is that of the first
  static_assert(8 * WAVES % 16 == 0, "");
  const int piece = (lane % 8) ^ ((8 * w + lrow) / 2 % 8);
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const bool left = i < LEFT;
    const int r = ((left ? i : i - LEFT) * WAVES + w) * 8 + lrow;
    const int most = (left ? p.M - m0 : p.N - n0) - 1;   // rows behind the end: the last one, not stored
    from[i] = (unsigned)(r < most ? r : most) * (unsigned)(left ? p.lda : p.ldb) + 16 * piece;
  }
  v4i held[WHOLE ? 1 : LOADS];   // without whole pieces: the next step's, on their way to LDS
  auto stage = [&](int kb, unsigned char* lds) {
    const bool full = (kb + 1) * kK <= p.K;
    const int k = kb * kK + 16 * piece;
    if constexpr (WHOLE) {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const unsigned char* at = (i < LEFT ? base_a : base_b) + kb * kK + from[i];
        if (!full) at = k < p.K ? at : reinterpret_cast<const unsigned char*>(kZeros);
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) void*)at,
            (__attribute__((address_space(3))) void*)(lds + (i * WAVES + w) * 1024), 16, 0, 0);
      }
    } else if (full) {   // pieces at any address
#pragma unroll
      for (int i = 0; i < LOADS; ++i)
        __builtin_memcpy(&held[i], (i < LEFT ? base_a : base_b) + kb * kK + from[i], 16);
    } else {
#pragma unroll
      for (int i = 0; i < LOADS; ++i)
        held[i] = piece16((i < LEFT ? base_a : base_b) + from[i] - 16 * piece, k, p.K);
    }
  };
  auto commit = [&](int kb, unsigned char* lds) {
    if constexpr (!WHOLE) {
      if ((kb + 1) * kK > p.K)
#pragma unroll
        for (int i = 0; i < LOADS; ++i) held[i] = piece_end(held[i], kb * kK + 16 * piece, p.K);
#pragma unroll
      for (int i = 0; i < LOADS; ++i)
        *reinterpret_cast<v4i*>(lds + (i * WAVES + w) * 1024 + lane * 16) = held[i];
    }
  };
  const int r16 = lane & 15, g = lane >> 4;
  const int piece0 = ((2 * g) ^ (r16 / 2)) * 16, piece1 = piece0 ^ 16;
  auto operand = [&](const unsigned char* lds, int row) {   // row: a multiple of 16
    const unsigned char* at = lds + (row + r16) * kK;
    v8i x;
    __builtin_memcpy(&x, at + piece0, 16);
    __builtin_memcpy((char*)&x + 16, at + piece1, 16);
    return x;
  };

  v4f acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  const unsigned char *sa[MT], *sb[NT];   // the scales of this lane's rows
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = m0 + wm + 16 * i + r16;
    sa[i] = p.sa + (long)(m < p.M ? m : p.M - 1) * steps;
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    int n = n0 + wn + 16 * j + r16;
    n = n < p.N ? n : p.N - 1;
    sb[j] = p.sb + (long)(p.square ? n / kGroup : n) * steps;
  }
  unsigned ea[MT], eb[NT], na[MT], nb[NT];   // of four steps, and of the next four
  auto step = [&](int kb, const unsigned char* here, unsigned char* there) {
    // this step's loads are done: those of the steps behind it may be on their way, at least LOADS a step
    if (DEEP && kb + 2 < steps) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * LOADS) : "memory");
    else if (DEEP && kb + 1 < steps) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if constexpr (DEEP) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();   // without a wait for all loads
      asm volatile("" ::: "memory");
    } else {
      __syncthreads();
    }
    if (kb % 4 == 0) {
      const int shift = scales_shift(kb, steps);
#pragma unroll
      for (int i = 0; i < MT; ++i) ea[i] = na[i] >> shift;
#pragma unroll
      for (int j = 0; j < NT; ++j) eb[j] = nb[j] >> shift;
      if (kb + 4 < steps) {
        scales4<MT>(sa, kb + 4, steps, na);
        scales4<NT>(sb, kb + 4, steps, nb);
      }
    }
    constexpr int ahead = DEEP ? 3 : 1;
    if (kb + ahead < steps) stage(kb + ahead, there);
    group_product<T, MT, NT>([&](int i) { return operand(here, wm + 16 * i); },
                             [&](int j) { return operand(here, BM + wn + 16 * j); }, ea, eb, acc);
    if (kb + 1 < steps) commit(kb + 1, there);
#pragma unroll
    for (int i = 0; i < MT; ++i) ea[i] >>= 8;
#pragma unroll
    for (int j = 0; j < NT; ++j) eb[j] >>= 8;
  };
  if (steps > 0) {
    scales4<MT>(sa, 0, steps, na);
    scales4<NT>(sb, 0, steps, nb);
    stage(0, lds0);
    commit(0, lds0);
  }
  if constexpr (DEEP) {
    if (steps > 1) stage(1, lds1);
    if (steps > 2) stage(2, lds2);
    for (int kb = 0; kb < steps; kb += 4) {
      step(kb, lds0, lds3);
      if (kb + 1 < steps) step(kb + 1, lds1, lds0);
      if (kb + 2 < steps) step(kb + 2, lds2, lds1);
      if (kb + 3 < steps) step(kb + 3, lds3, lds2);
    }
  } else {
    for (int kb = 0; kb < steps; kb += 2) {
      step(kb, lds0, lds1);
      if (kb + 1 < steps) step(kb + 1, lds1, lds0);
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
      store4((T*)p.out, p.ldo, m0 + wm + 16 * i + r16, n0 + wn + 16 * j + 4 * g, p.M, p.N, acc[i][j]);
}

// Few rows of out (M <= 16 MT): bound by B's bytes.  A block takes 16 columns of out; its waves share
// out the groups along K, each by itself and without barriers, up to three groups on their way to
// its own part of LDS, and their sums are added up in a fixed order.  (Operands
// read to registers take a cache access for every 16 bytes, since neighbouring lanes hold different
// rows: 32 x 6144 x 4096 18.3 us against 11.7.)
template <typename T, int MT, int WAVES, bool WHOLE>
__global__ __launch_bounds__(64 * WAVES) void matmul_few_kernel(const MatmulArgs p) {
  constexpr int LOADS = 2 * (MT + 1), BYTES = LOADS * 1024;
  __shared__ __attribute__((aligned(16))) unsigned char lds0[WAVES * BYTES], lds1[WAVES * BYTES],
      lds2[WAVES * BYTES];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int groups = (p.K + kK - 1) / kK, n0 = blockIdx.x * 16;
  const int mine = groups > w ? (groups - w + WAVES - 1) / WAVES : 0;   // groups w, w + WAVES, ...

  // rows of a group's loads: A's 16 MT, then B's 16; those behind the end: the last one, not stored
  const unsigned char* row[LOADS];
  const int piece = (lane % 8) ^ (lane / 8 / 2 % 8);   // of even loads; of odd ones, whose rows are 8 on, ^ 4
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const bool left = i < 2 * MT;
    const int r = (left ? i : i - 2 * MT) * 8 + lane / 8, most = (left ? p.M : p.N - n0) - 1;
    const int at = r < most ? r : most;
    row[i] = left ? p.a + (long)at * p.lda : p.b + (long)(n0 + at) * p.ldb;
  }
  const unsigned char* srow[MT + 1];   // the scales of this lane's rows, B's last
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = 16 * i + r16 < p.M ? 16 * i + r16 : p.M - 1;
    srow[i] = p.sa + (long)m * groups;
  }
  const int n = n0 + r16 < p.N ? n0 + r16 : p.N - 1;
  srow[MT] = p.sb + (long)(p.square ? n / kGroup : n) * groups;

  v4f acc[MT][1];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i][0] = v4f{0.f, 0.f, 0.f, 0.f};
  v4i held[WHOLE ? 1 : LOADS];
  unsigned e0[MT + 1], e1[MT + 1], e2[MT + 1];
  auto stage = [&](int j, unsigned char* lds, unsigned (&e)[MT + 1]) {
    if (j >= mine) return;
    // the reads of what lay there are done before anything else comes there
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const int kb = w + j * WAVES;
    const bool full = (kb + 1) * kK <= p.K;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int k = kb * kK + 16 * (i % 2 ? piece ^ 4 : piece);
      if constexpr (WHOLE) {
        const unsigned char* at = row[i] + k;
        if (!full) at = k < p.K ? at : reinterpret_cast<const unsigned char*>(kZeros);
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) void*)at,
            (__attribute__((address_space(3))) void*)(lds + w * BYTES + i * 1024), 16, 0, 0);
      } else if (full) {
        __builtin_memcpy(&held[i], row[i] + k, 16);
      } else {
        held[i] = piece16(row[i], k, p.K);
      }
    }
    if constexpr (!WHOLE)
      if (!full)
#pragma unroll
        for (int i = 0; i < LOADS; ++i) held[i] = piece_end(held[i], kb * kK + 16 * (i % 2 ? piece ^ 4 : piece), p.K);
#pragma unroll
    for (int i = 0; i <= MT; ++i) e[i] = srow[i][kb];
    if constexpr (!WHOLE)
#pragma unroll
      for (int i = 0; i < LOADS; ++i)
        *reinterpret_cast<v4i*>(lds + w * BYTES + i * 1024 + lane * 16) = held[i];
  };
  auto step = [&](int j, const unsigned char* lds, const unsigned (&e)[MT + 1]) {
    if (j >= mine) return;
    auto operand = [&](int tile) {
      const unsigned char* at = lds + w * BYTES + (tile * 16 + r16) * kK;
      v8i x;
      __builtin_memcpy(&x, at + ((2 * g) ^ (r16 / 2)) * 16, 16);
      __builtin_memcpy((char*)&x + 16, at + ((2 * g + 1) ^ (r16 / 2)) * 16, 16);
      return x;
    };
    unsigned ea[MT], eb[1] = {e[MT]};
#pragma unroll
    for (int i = 0; i < MT; ++i) ea[i] = e[i];
    group_product<T, MT, 1>([&](int i) { return operand(i); }, [&](int) { return operand(MT); }, ea, eb, acc);
  };
  stage(0, lds0, e0);
  stage(1, lds1, e1);
  stage(2, lds2, e2);
  for (int j = 0; j < mine; j += 3) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // three groups are there
    step(j, lds0, e0);
    stage(j + 3, lds0, e0);
    step(j + 1, lds1, e1);
    stage(j + 4, lds1, e1);
    step(j + 2, lds2, e2);
    stage(j + 5, lds2, e2);
  }
  // the sums: of tile i by wave i
  v4f(*sums)[MT][64] = reinterpret_cast<v4f(*)[MT][64]>(lds0);
  static_assert(WAVES * MT * 64 * 16 <= WAVES * BYTES, "");
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MT; ++i) sums[w][i][lane] = acc[i][0];
  __syncthreads();
  for (int i = w; i < MT; i += WAVES) {
    v4f c = sums[0][i][lane];
#pragma unroll
    for (int q = 1; q < WAVES; ++q) c += sums[q][i][lane];
    store4((T*)p.out, p.ldo, 16 * i + r16, n0 + 4 * g, p.M, p.N, c);
  }
}

namespace {

template <typename T, int BM, int BN, int WM, int WN>
hipError_t tiles(const MatmulArgs& a, bool whole, hipStream_t s) {
  const long n = (long)((a.N + BN - 1) / BN) * ((a.M + BM - 1) / BM);
  const unsigned grid = (unsigned)((n + 7) / 8 * 8);
  constexpr int threads = (BM / WM) * (BN / WN) * 64;
  if (whole) matmul_kernel<T, BM, BN, WM, WN, true, BM == 64><<<grid, threads, 0, s>>>(a);
  else if constexpr (BM <= 128) matmul_kernel<T, BM, BN, WM, WN, false, false><<<grid, threads, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, int MT, int WAVES>
hipError_t few(const MatmulArgs& a, bool whole, hipStream_t s) {
  const unsigned grid = (unsigned)((a.N + 15) / 16);
  if (whole) matmul_few_kernel<T, MT, WAVES, true><<<grid, 64 * WAVES, 0, s>>>(a);
  else matmul_few_kernel<T, MT, WAVES, false><<<grid, 64 * WAVES, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t matmul(const MatmulArgs& a, hipStream_t s) {
  const bool whole = ((reinterpret_cast<uintptr_t>(a.a) | reinterpret_cast<uintptr_t>(a.b) |
                       (uintptr_t)a.lda | (uintptr_t)a.ldb | (uintptr_t)a.K) & 15) == 0;
  // Few rows: eight waves a block (four for more than 32 rows) while there is a block of 16 columns a CU at
  // most; half as many above, so that two blocks share a CU's LDS: bf16, K = 4096, us, 32 x 6144 10.1,
  // as before 11.4, 32 x 16384 20.3 and 23.7, 64 x 6144 14.8 and 16.7; the other way round 32 x 4096
  // with K = 16384 20.1, with four waves 21.1.  Above two blocks a CU, more than 32 rows are faster by
  // tiles of 64: 64 x 8192 15.2, tiles 16.8; 64 x 12288 27.3 and 17.5.
  if (a.M <= (a.N <= 32 * 256 ? 64 : 32)) {
    if (a.N <= 16 * 256)
      return a.M <= 16 ? few<T, 1, 8>(a, whole, s) : a.M <= 32 ? few<T, 2, 8>(a, whole, s) : few<T, 4, 4>(a, whole, s);
    return a.M <= 16 ? few<T, 1, 4>(a, whole, s) : a.M <= 32 ? few<T, 2, 4>(a, whole, s) : few<T, 4, 2>(a, whole, s);
  }
  // Tiles of 128 where they fill the CUs, of 64 below (bf16, K = 4096, us): 512 x 4096, 128 tiles, 64
  // 23.9, 128 33.2; 1024 x 4096, 256 tiles, 64 36.6, 128 35.6; 2048 x 4096 66.1 and 47.7.  Tiles of 256,
  // whose operands are read from LDS half as often, one a CU: a round of them takes what 5 / 3 rounds
  // of 128, two a CU, do: 8192 x 2048 256 72.4, 128 82.3; 3000 x 4096 71.3 and 81.9; 4096 x 6144 (384
  // tiles, two rounds) 138 and 124; 2048 x 4096 70.2 and 47.7.  Their float32 form spills.
  auto blocks = [&](int bm, int bn) { return (long)((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn); };
  const long half = blocks(128, 128);
  if constexpr (sizeof(T) == 2)
    if (whole && (blocks(256, 256) + 255) / 256 * 5 <= (half + 511) / 512 * 3)
      return tiles<T, 256, 256, 64, 128>(a, true, s);
  if (half >= 256) return tiles<T, 128, 128, 64, 64>(a, whole, s);
  return tiles<T, 64, 64, 32, 32>(a, whole, s);
}

}  // namespace

hipError_t launch_matmul(const MatmulArgs& a, int dtype, hipStream_t s) {
  if (dtype == S4DPLR_F32) return matmul<float>(a, s);
  return dtype == S4DPLR_BF16 ? matmul<bf16>(a, s) : matmul<f16>(a, s);
}

}  // namespace s4
