// Root-mean-square norm: arguments of the launchers.
#pragma once

#include <hip/hip_runtime_api.h>

#include "s4dplr.h"

namespace s4 {

struct RmsArgs {
  const void *x, *residual;   // residual may be NULL
  const float* gamma;         // may be NULL: 1
  void *h, *y;                // each may be NULL
  unsigned char *q, *scales;  // both or none
  float* rstd;                // written forward (may be NULL), read backward
  const void *dy, *dh;        // backward; dh may be NULL
  void* dx;
  float *dgamma, *part;
  long rows, D;
  float eps;
};

hipError_t launch_rms_fwd(const RmsArgs& a, int dtype, hipStream_t s);
hipError_t launch_rms_bwd(const RmsArgs& a, int dtype, hipStream_t s);

}  // namespace s4
