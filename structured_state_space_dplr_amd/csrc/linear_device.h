// Device side of linear attention's chunked pass.  The products run on the bf16 matrix
// cores; an operand is a sum of bf16 parts (delta_device.h), so that fp32 accuracy is kept.
#pragma once

#include "delta_device.h"
#include "linear.h"

namespace s4 {

constexpr LinRows lin_rows(long tokens, int each, const int* offsets, int s, int a, int b) {
  if (!offsets) return LinRows{(long)each * s, each};
  const Rows r = clamp_rows((int)tokens, a, b);
  return LinRows{r.start, r.len};
}
template <typename A>
__device__ __forceinline__ LinRows lin_rows(const A& p, int s) {
  return p.offsets ? lin_rows(p.tokens, p.each, p.offsets, s, p.offsets[s], p.offsets[s + 1])
                   : LinRows{(long)p.each * s, p.each};
}

// The sequence whose segments include `slot`, by all lanes of a wave together: the last whose
// first slot is at most `slot`, 64 sequences probed at a time.
template <typename A>
__device__ __forceinline__ int lin_sequence(const A& p, long slot) {
  const int lane = threadIdx.x & 63;
  int s = 0;
  for (int n = p.sequences;;) {   // sequences s .. s + n are left
    const int step = (n + 63) / 64, at = lane * step;
    const bool le = at < n && lin_rows(p, s + at).slot(s + at, p.segment) <= slot;
    const int c = __popcll(__ballot(le));
    if (c == 0) return s;
    s += (c - 1) * step;
    n -= (c - 1) * step;
    if (step == 1) return s;
    n = n < step ? n : step;
  }
}

// Item -> rows of a block's work: items below `sequences` are sequences of one segment, the
// others slots.
struct LinItem {
  int s, m, of;     // sequence, segment, number of segments (0: one that has no slot)
  long slot, start;
  int len;
};
// The same value, for all that the compiler knows another one: a load of it is not put under the
// condition under which it is used, where it would be waited for at once.
__device__ __forceinline__ void touch(float& v) { asm volatile("" : "+v"(v)); }

// The thread's number, not known to be the one of another call: what is computed from it is
// computed there, and not kept in registers through a loop (64 of which would be spilled).
__device__ __forceinline__ unsigned thread() {
  unsigned t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

__device__ __forceinline__ long uniform(long v) {
  return (long)(unsigned)__builtin_amdgcn_readfirstlane((int)v) |
         (long)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32;
}
template <typename A>
__device__ __forceinline__ bool find_item(const A& p, long item, LinItem* w) {
  if (item < p.sequences) {
    const LinRows r = lin_rows(p, (int)item);
    if (r.len > p.segment) return false;
    *w = LinItem{(int)item, 0, 0, -1, r.start, (int)r.len};
    return true;
  }
  const long slot = item - p.sequences;
  if (slot >= p.slots) return false;
  const int s = lin_sequence(p, slot);
  const LinRows r = lin_rows(p, s);
  const long m = slot - r.slot(s, p.segment);
  const int of = r.segments(p.segment);
  if (r.len <= p.segment || m < 0 || m >= of) return false;
  const long left = r.len - m * p.segment;
  *w = LinItem{s, (int)m, of, slot, r.start + m * p.segment, (int)(left < p.segment ? left : p.segment)};
  return true;
}

// The item's rows, known to be the same for all lanes.
template <typename A>
__device__ __forceinline__ bool lin_item(const A& p, long item, LinItem* w) {
  LinItem t = {};
  const bool found = find_item(p, item, &t);
  *w = LinItem{__builtin_amdgcn_readfirstlane(t.s), __builtin_amdgcn_readfirstlane(t.m),
               __builtin_amdgcn_readfirstlane(t.of), uniform(t.slot), uniform(t.start),
               __builtin_amdgcn_readfirstlane(t.len)};
  return __builtin_amdgcn_readfirstlane(found) != 0;
}

}  // namespace s4
