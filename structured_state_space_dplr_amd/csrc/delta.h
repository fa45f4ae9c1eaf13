// Gated delta rule: the plan, the layout of its buffers and the launchers.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstddef>

#include "s4dplr.h"

namespace s4 {
constexpr int kChunk = 64;    // tokens a chunk
constexpr int kFrag = 1024;   // bytes of one matrix-instruction operand: 64 lanes x 8 bf16
}  // namespace s4

struct s4dplr_delta_plan {
  int sequences;
  long tokens;
  int each;     // tokens / sequences
  int Hk, Hv, dk, dv;
  int dtype;
  bool training;
  int dkp;      // dk rounded up to 64, 128 or 256
  int parts;    // bf16 parts an input element is the exact sum of: 1 (bf16), 2 (fp16), 3 (fp32)
  long slots;   // chunks of all sequences, at most
  // Workspace, byte offsets.  "frags" are operands in the register order of the
  // 16x16x32 bf16 matrix instruction, [part][row tile][k step] of kFrag bytes.
  size_t off_k, off_q;       // [slot][Hk] frags of K, Q (64 x dk)
  size_t off_kt, off_qt;     // [slot][Hk] frags of K^T, Q^T (dk x 64); Q^T backward only
  size_t off_x, off_p;       // [slot][Hv] frags of (I + H diag beta)^-1 and of scale P (64 x 64);
                             // backward: of their transposes
  size_t off_vec;            // [slot][Hv] DeltaVec
  size_t off_dv, off_ds;     // backward: [slot][Hv] fp32 dV [64][dv], dS' [dk][dv]
  size_t off_gates;          // backward, dk > 64: [ceil(dk / 64)][2][tokens][Hv] fp32 parts of dg, dbeta
  size_t total;
  // saved (training): [slot][Hv] fp32 N [64][dv], S [dk][dv] (the state before the chunk)
  size_t off_n, off_s;
  size_t saved_total;
};

namespace s4 {

// Per chunk and value head; rows behind the sequence's end have beta = 0 and the
// decay of the last row.
struct DeltaVec {
  float e[kChunk];      // 2^G_i
  float d[kChunk];      // 2^(G_last - G_i)
  float beta[kChunk];
  double G[kChunk];     // inclusive sums of g / log 2 over the chunk
};

struct DeltaArgs {
  const void *q, *k, *v;
  long ldq, ldk, ldv;         // elements from one token to the next
  const float *g, *beta;
  const int* offsets;         // [sequences + 1], or NULL: equal lengths
  const float* state;         // may be NULL: zeros
  void* o;
  float* state_out;           // may be NULL
  float scale;
  const void* dout;           // backward
  const float* dstate_out;    // backward, may be NULL: zeros
  void *dq, *dk, *dv;
  float *dg, *dbeta;
  float* dstate;              // may be NULL
  unsigned char *ws, *saved;
  int step_tokens;            // sequences of at most so many tokens go token by token
  int least;                  // max(1, step_tokens + 1)
};

// Longest sequence that is taken token by token.  In bf16 a token costs 1.4 us (128 sequences,
// 16 heads of 128 x 128: 14 us), a chunk with its preparation what 9 to 16 tokens do.  Token by
// token against by chunks, 16 heads of 128 x 128: one sequence, 8 tokens 15.5 us against
// 16.9, 12 tokens 21.2 against 16.9; 16 sequences, 16 tokens 43.3 against 43.6, 24 tokens 60.4
// against 43.7; 128 sequences, 16 tokens 255 against 270, 24 tokens 370 against 276.  (8 heads of
// 64 x 64, 128 sequences: 16 tokens 66 against 81, 24 tokens 95 against 81.)  The line is
// drawn where the chunked form's blocks (16 columns each) fill the 256 CUs.  It holds for all
// types, though a chunk costs more in fp16 and fp32: 128 sequences of 24 tokens 367 against 459
// in fp16, 335 against 575 in fp32, one sequence of 12 tokens 18.4 against 20.0 in fp32.
inline int step_limit(const s4dplr_delta_plan* p) {
  return (long)p->sequences * p->Hv * ((p->dv + 15) / 16) > 256 ? 16 : 8;
}

// Where a sequence lies in the packed rows, and its chunks in the slots.  `least` is the
// shortest length that a call takes by chunks.  Chunks of sequence s are slots
//   first(s) = floor(start / 64) + min(s, floor(start / least))
// and on: disjoint for any lengths, since ceil((b - a) / 64) <= floor(b / 64) - floor(a / 64) + 1
// and the second term grows behind every sequence of `least` tokens or more; and below
// floor(tokens / 64) + min(sequences, floor(tokens / least)).
struct Rows {
  long start, len;
  constexpr long first(int s, int least) const {
    const long before = start / least;
    return start / kChunk + (s < before ? s : before);
  }
  constexpr int chunks() const { return (int)((len + kChunk - 1) / kChunk); }
};
// The sequence from row a to row b of n.  Offsets outside [0, n] and falling ones, whatever
// their values, are clamped before they are subtracted: no access leaves the buffers.
constexpr Rows clamp_rows(int n, int a, int b) {
  const int start = a < 0 ? 0 : a > n ? n : a, end = b < start ? start : b > n ? n : b;
  return Rows{start, end - start};
}

// Whether a packed call without `saved` takes its short sequences token by token, in a
// launch of their own.  The lengths are known to the device only.  Where sequences are short
// in the mean, both forms run, each on its own sequences; else all go by chunks, which one
// more launch for the few short ones would not make faster.
inline bool packed_steps(const s4dplr_delta_plan* p) {
  return p->tokens <= (long)step_limit(p) * p->sequences;
}
// Slots that the plan's calls need, at most.
inline long chunk_slots(const s4dplr_delta_plan* p) {
  const long most = p->tokens / (p->training || !packed_steps(p) ? 1 : step_limit(p) + 1);
  return p->tokens / kChunk + (p->sequences < most ? p->sequences : most);
}

hipError_t launch_delta_steps(const s4dplr_delta_plan* p, const DeltaArgs& a, hipStream_t s);
hipError_t launch_delta_prep(const s4dplr_delta_plan* p, const DeltaArgs& a, bool bwd,
                             hipStream_t s);
hipError_t launch_delta_scan(const s4dplr_delta_plan* p, const DeltaArgs& a, hipStream_t s);
hipError_t launch_delta_scan_bwd(const s4dplr_delta_plan* p, const DeltaArgs& a, hipStream_t s);
hipError_t launch_delta_grads(const s4dplr_delta_plan* p, const DeltaArgs& a, hipStream_t s);

}  // namespace s4
