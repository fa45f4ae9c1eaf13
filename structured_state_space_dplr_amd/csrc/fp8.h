// Quantization to 8 bits and the 8-bit matrix product: arguments of the launchers.
#pragma once

#include <hip/hip_runtime_api.h>

#include "s4dplr.h"

namespace s4 {

struct QuantizeArgs {
  const void* x;
  long ldx;                          // elements from one row to the next
  unsigned char *q, *scales;         // [rows][cols] and its scales, or NULL
  unsigned char *qt, *scales_t;      // [cols][rows] and its scales, or NULL
  int rows, cols;
  bool square;                       // one scale for 128 x 128 values
};

struct MatmulArgs {
  const unsigned char *a, *sa, *b, *sb;
  long lda, ldb, ldo;
  void* out;
  int M, N, K;
  bool square;                       // sb is [ceil(N / 128)][ceil(K / 128)]
};

hipError_t launch_quantize(const QuantizeArgs& a, int dtype, hipStream_t s);
hipError_t launch_matmul(const MatmulArgs& a, int dtype, hipStream_t s);

}  // namespace s4
