// Layer norm: arguments of the launchers and the split of the backward pass.
#pragma once

#include <hip/hip_runtime_api.h>

#include "s4dplr.h"

namespace s4 {

constexpr long kNormMaxD = 32768;      // a row of 16 waves, 32 values a lane
// Blocks of the forward pass over rows: eight a CU (16: 8192 x 8192 bf16 45.1 -> 50.5 us,
// and no row gains over 5 %); two of 16 waves.
constexpr long kNormBlocks = 2048;

constexpr long kNormChannels = 256;    // channels whose sums stay in registers

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
// per tile of work (a row, 4 rows up to 512 values, or 64 positions) up to two a CU, one for
// rows above 2048 values and for channels above 64, whose blocks keep more loads on
// their way.  More blocks cost more traffic of partial sums, fewer leave the memory
// idle.  Whole calls, with the partial rows' sum: 16384 x 2048 bf16 51.4 us with eight a CU, 41.9
// with four, 42.6 with two (half the workspace), 51.2 with one; 16384 x 4096 92.7 with four, 80.1
// with two, 76.7 with one; 4096 x 4096 30.6, 25.3 and 24.3; channels of 32 x 256 x 1024
// fp32 30.2 with two, 25.4 with one.  Above 16384 values or kNormChannels channels the
// columns' sums have their own kernel, whose blocks take some columns each.
inline long norm_parts(long outer, long D, long inner) {
  const long tiles = inner > 1 ? (outer * inner + 63) / 64 : D <= 512 ? (outer + 3) / 4 : outer;
  const long most = inner > 1 ? (D > kNormChannels ? 64 : D > 64 ? 256 : 512) : D > 16384 ? 32 : D > 2048 ? 256 : 512;
  return tiles < 1 ? 1 : tiles < most ? tiles : most;
}

hipError_t launch_norm_fwd(const NormArgs& a, int dtype, hipStream_t s);
hipError_t launch_norm_bwd(const NormArgs& a, int dtype, hipStream_t s);

}  // namespace s4
