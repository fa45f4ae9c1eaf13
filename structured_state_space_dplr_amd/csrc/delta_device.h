// Device side shared by the chunked gated delta rule's kernels.
//
// The matrix products run on the bf16 matrix cores.  An operand enters as a sum
// of bf16 parts (hi, mid, lo: 8 significant bits each), so a bf16 input is one
// part, fp16 two, fp32 three; values computed on the way (states, the inverse, the
// pairs' products, corrections) take three, which keeps fp32 accuracy (the dropped cross
// products are below 2^-24 relative), so 16-bit outputs are those of fp32 tensors of the same
// values, rounded once.  Three parts of products cost 6 matrix instructions where the fp32
// instruction would take 16 times the bf16 one's time.
#pragma once

#include "delta.h"
#include "vec.h"

// for pointers whose address space the compiler does not find out by itself
#define GLOBAL __attribute__((address_space(1)))

namespace s4 {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

// 16x16x32: lane l holds row (A) or column (B) l % 16, k = 8 (l / 16) .. + 8; the
// result's column l % 16, rows 4 (l / 16) .. + 4.
__device__ __forceinline__ v4f mfma(v8bf a, v8bf b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// 16x16x4 fp32: lane l holds row / column l % 16, k = l / 16.
__device__ __forceinline__ v4f mfma32(float a, float b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// c += a b over the parts, without the products of weight below KEEP parts.
template <int KEEP, int PA, int PB>
__device__ __forceinline__ v4f mfma_parts(const v8bf (&a)[PA], const v8bf (&b)[PB], v4f c) {
#pragma unroll
  for (int i = PA - 1; i >= 0; --i)
#pragma unroll
    for (int j = PB - 1; j >= 0; --j)
      if (i + j < KEEP) c = mfma(a[i], b[j], c);
  return c;
}

typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// P bf16 parts whose sum is x (exactly, with three parts), by pairs: the hardware
// converts two values an instruction.
template <int P>
__device__ __forceinline__ void split2(v2f x, v2bf (&out)[P]) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    out[p] = __builtin_convertvector(x, v2bf);
    if (p + 1 < P) x -= __builtin_convertvector(out[p], v2f);
  }
}
template <int P>
__device__ __forceinline__ void split8(const float* x, v8bf (&out)[P]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    v2bf t[P];
    split2<P>(v2f{x[i], x[i + 1]}, t);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      out[p][i] = t[p][0];
      out[p][i + 1] = t[p][1];
    }
  }
}
template <int P>
__device__ __forceinline__ void split4(v4f x, v4bf (&out)[P]) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    v2bf t[P];
    split2<P>(v2f{x[i], x[i + 1]}, t);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      out[p][i] = t[p][0];
      out[p][i + 1] = t[p][1];
    }
  }
}

// Eight elements of one row, zero behind the first n.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, float* out) {
  if (n >= 8) {
    T t[8];
    __builtin_memcpy(t, p, sizeof(t));
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = to_f32(t[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = i < n ? to_f32(p[i]) : 0.f;
  }
}

// Eight floats, the first n of them.
__device__ __forceinline__ void store8(float* p, int n, const float* x) {
  if (n >= 8) {
    __builtin_memcpy(p, x, 32);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = x[i];
  }
}

// LDS written by one lane of a wave is read by another behind this
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Operand `frag` (a constant) behind a uniform base; off = 16 lane.  The base takes
// the multiples of 4 KB, so scalar registers and the instruction's own offset hold
// the rest of the address.
__device__ __forceinline__ v8bf load_frag(const unsigned char* base, int frag, unsigned off) {
  return *reinterpret_cast<const v8bf*>(base + (size_t)(frag & ~3) * kFrag + (off + (frag & 3) * kFrag));
}

// Operand of 16 columns (the fast index of m [part][ROWS][LD] in LDS) by 32 k (its rows r0
// ..): lane (lr, lg) gets its column, rows r0 + 8 lg .. + 8.  In the transposing read 16
// lanes fetch 4 rows of 4 groups of 4 columns, and lane i receives column i of the
// 16.  The groups are STEP columns apart: 4, or 8 for tiles of dk in the order of K^T's
// rows.
template <int P, int STEP, int ROWS, int LD>
__device__ __forceinline__ void get_tr(const __bf16 (*m)[ROWS][LD], int r0, int c0, int lr, int lg,
                                       v8bf (&out)[P]) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) v4s lds4;
#pragma unroll
  for (int q = 0; q < P; ++q) {
    const __bf16* a = &m[q][r0 + 8 * lg + (lr >> 2)][c0 + STEP * (lr & 3)];
    union {
      v4s h[2];
      v8bf v;
    } u;
    u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)a);
    u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(a + 4 * LD));
    out[q] = u.v;
  }
}

// 2^x for a difference x held in 64 bits, at fp32 accuracy for any size of it: the
// hardware's 2^f for |f| <= 1 / 2, scaled by the whole part.
__device__ __forceinline__ float exp_diff(double x) {
  const double n = __builtin_rint(x);
  return ldexpf(__builtin_amdgcn_exp2f((float)(x - n)), (int)n);
}

__device__ __forceinline__ Rows rows_of(const s4dplr_delta_plan& p, const int* offsets, int s) {
  if (!offsets) return Rows{(long)p.each * s, p.each};
  return clamp_rows((int)p.tokens, offsets[s], offsets[s + 1]);
}

// Block -> (sequence and head, slice of the dv columns).  Blocks go round robin
// over the 8 XCDs; the slices of one head read the same operands, so they take
// ids that are equal modulo 8 and share one L2.
__device__ __forceinline__ bool slice_of(int heads, int slices, int* head, int* slice) {
  const int b = blockIdx.x, g = b >> 3;
  *head = (g / slices) * 8 + (b & 7);
  *slice = g % slices;
  return *head < heads;
}

// The sequence whose chunks include `slot`, by all lanes of a wave together: the last
// with first(s) <= slot, 64 sequences probed at a time (first(s) rises with s; for
// offsets out of order some sequence is returned, and the caller's bounds hold).
__device__ __forceinline__ int sequence_of(const s4dplr_delta_plan& p, const DeltaArgs& a,
                                           long slot) {
  const int lane = threadIdx.x & 63;
  int s = 0;
  for (int n = p.sequences;;) {   // sequences s .. s + n are left
    const int step = (n + 63) / 64, at = lane * step;
    const bool le = at < n && rows_of(p, a.offsets, s + at).first(s + at, a.least) <= slot;
    const int c = __popcll(__ballot(le));
    if (c == 0) return s;
    s += (c - 1) * step;
    n -= (c - 1) * step;
    if (step == 1) return s;
    n = n < step ? n : step;
  }
}

}  // namespace s4
