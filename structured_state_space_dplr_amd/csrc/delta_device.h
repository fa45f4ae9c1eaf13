// Device side shared by the chunked gated delta rule's kernels.
//
// The matrix products run on the bf16 matrix cores.  An operand enters as a sum
// of bf16 parts (hi, mid, lo: 8 significant bits each), so a bf16 input is one
// part, fp16 two, fp32 three; values computed on the way (states, the inverse,
// corrections) take three parts wherever they reach the carried state or an
// fp32 output, which keeps those at fp32 accuracy (the dropped cross products are
// below 2^-24 relative), and two (2^-16) where the only reader is an output of
// 16 bits.  Three parts of products cost 6 matrix instructions where the fp32
// instruction would take 16 times the bf16 one's time.
#pragma once

#include "delta.h"
#include "vec.h"

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

template <int P>
__device__ __forceinline__ void split8(const float* x, v8bf (&out)[P]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float r = x[i];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const __bf16 h = (__bf16)r;
      out[p][i] = h;
      r -= (float)h;
    }
  }
}
template <int P>
__device__ __forceinline__ void split4(v4f x, v4bf (&out)[P]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float r = x[i];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const __bf16 h = (__bf16)r;
      out[p][i] = h;
      r -= (float)h;
    }
  }
}

// Eight elements of one row, zero behind `n`.
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

// LDS written by one lane of a wave is read by another behind this
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ v8bf load_frag(const unsigned char* base, int frag, int lane) {
  return *reinterpret_cast<const v8bf*>(base + (size_t)frag * kFrag + lane * 16);
}

// exp of a difference held in 64 bits, at fp32 accuracy for any size of it
__device__ __forceinline__ float exp_diff(double x) {
  const float h = (float)x;
  return h > -126.f ? expf(h) * (1.f + (float)(x - (double)h)) : expf(h);
}

// Where a sequence lies in the packed rows, and its chunks in the slots.  Chunks
// of sequence s are slots first(s) = floor(start / 64) + s and on: disjoint for
// any lengths, since ceil((b - a) / 64) <= floor(b / 64) - floor(a / 64) + 1.
// Offsets outside [0, tokens] or falling ones are clamped, so no access leaves
// the buffers.
struct Rows {
  long start, len;
  __device__ __forceinline__ long first(int s) const { return start / kChunk + s; }
  __device__ __forceinline__ int chunks() const { return (int)((len + kChunk - 1) / kChunk); }
};
__device__ __forceinline__ Rows rows_of(const int* offsets, long tokens, int sequences, int s) {
  Rows r;
  if (!offsets) {
    r.len = tokens / sequences;
    r.start = r.len * s;
    return r;
  }
  const long a = offsets[s], b = offsets[s + 1];
  r.start = a < 0 ? 0 : a > tokens ? tokens : a;
  r.len = (b > tokens ? tokens : b) - r.start;
  if (r.len < 0) r.len = 0;
  return r;
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

// The sequence whose chunks include `slot`, by all lanes of a wave together:
// sequences with first(s) <= slot are counted.
__device__ __forceinline__ int sequence_of(const int* offsets, long tokens, int sequences,
                                           long slot) {
  const int lane = threadIdx.x & 63;
  int n = 0;
  for (int s0 = 0; s0 < sequences; s0 += 64) {
    const int s = s0 + lane;
    const bool le = s < sequences && rows_of(offsets, tokens, sequences, s).first(s) <= slot;
    const int c = __popcll(__ballot(le));
    n += c;
    if (c < 64) break;
  }
  return n > 0 ? n - 1 : 0;
}

}  // namespace s4
