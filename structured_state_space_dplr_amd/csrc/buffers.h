// Checks of arguments that the token-major operators' entry points share.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstddef>
#include <cstdint>

#include "internal.h"
#include "s4dplr.h"

namespace s4 {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline bool valid_dtype(int d) { return d == S4DPLR_F32 || d == S4DPLR_BF16 || d == S4DPLR_F16; }
inline size_t elem(int dtype) { return dtype == S4DPLR_F32 ? 4 : 2; }

// A buffer of the call: address, bytes, bytes its address is a multiple of.
struct Buf {
  const void* p;
  size_t n, align;
};

inline bool overlaps(const Buf& a, const Buf& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.n && b0 < a0 + a.n;
}

// Every buffer aligned; every output apart from every input and from the other
// outputs.  `same`: an output that may be exactly the input `same_in`.
template <size_t NI, size_t NO>
s4dplr_status check_buffers(const Buf (&in)[NI], const Buf (&out)[NO], int same, int same_in) {
  for (const Buf& b : in)
    if (reinterpret_cast<uintptr_t>(b.p) % b.align) return S4DPLR_ERR_ALIGN;
  for (const Buf& b : out)
    if (reinterpret_cast<uintptr_t>(b.p) % b.align) return S4DPLR_ERR_ALIGN;
  for (size_t i = 0; i < NO; ++i) {
    for (size_t j = 0; j < NI; ++j) {
      if ((int)i == same && (int)j == same_in && out[i].p == in[j].p) continue;
      if (overlaps(out[i], in[j])) return S4DPLR_ERR_ALIAS;
    }
    for (size_t j = 0; j < i; ++j)
      if (overlaps(out[i], out[j])) return S4DPLR_ERR_ALIAS;
  }
  return S4DPLR_OK;
}

inline s4dplr_status done(hipError_t e) { return e == hipSuccess ? S4DPLR_OK : hip_failure(e); }

}  // namespace s4
