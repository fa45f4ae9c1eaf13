// Layer norm: arguments of the launchers and the split of the backward pass.
#pragma once

#include <hip/hip_runtime_api.h>

#include "s4dplr.h"

namespace s4 {

constexpr long kNormMaxD = 32768;      // a row of 16 waves, 32 values a lane
constexpr long kNormParts = 512;       // blocks of the backward pass: two per CU

struct NormArgs {
  const void* x;
  const float *gamma, *beta;
  void* y;
  float *mean, *rstd;   // written forward, read backward
  const void* dy;
  void* dx;
  float *dgamma, *dbeta, *part;
  long outer, D, inner;
  float eps;
};

// Blocks of the backward pass, the rows of its partial sums [2][parts][D]: one
// per tile of work (4 rows, or 64 positions) up to kNormParts.
inline long norm_parts(long outer, long inner) {
  const long tiles = inner == 1 ? (outer + 3) / 4 : (outer * inner + 63) / 64;
  return tiles < 1 ? 1 : tiles < kNormParts ? tiles : kNormParts;
}

hipError_t launch_norm_fwd(const NormArgs& a, int dtype, hipStream_t s);
hipError_t launch_norm_bwd(const NormArgs& a, int dtype, hipStream_t s);

}  // namespace s4
