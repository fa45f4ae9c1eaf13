// Linear attention's chunked pass for bf16 tensors.
#include "linear_pass.h"

namespace s4 {

hipError_t linear_pass_bf16(const LinPass& a, bool sum, hipStream_t s) {
  if (sum) return linear_launch<bf16, 1, kSum>(a, s);
  // out of the pass, if any, in the tensors' type, without sums by rows
  const bool plain = !a.out_f32 && !a.dot;
  return plain ? linear_launch<bf16, 1, kOut>(a, s) : linear_launch<bf16, 1, kGrad>(a, s);
}

int linear_parts_bf16(int dx, int dw) {
  int parts = 0;
  linear_shape<1>(dx, dw, [&](auto, auto waves, auto cw, auto) {
    constexpr int W = decltype(waves)::value, COLS = W * decltype(cw)::value;
    parts = (dw + COLS - 1) / COLS * W;
  });
  return parts;
}

}  // namespace s4
