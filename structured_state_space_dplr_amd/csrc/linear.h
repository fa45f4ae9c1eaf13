// Linear attention with decay: the plan, the layout of its buffers and the launchers.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstddef>

#include "s4dplr.h"

struct s4dplr_linear_attention_plan {
  int sequences;
  long tokens;
  int each;     // tokens / sequences
  int Hk, Hv, dk, dv;
  int dtype;
  bool training;
  // Sequences of more than `segment` rows are cut into segments of so many, each a block's
  // work; the states between them have slots.  Segments of sequence s are slots
  //   floor(start / segment) + min(s, floor(start / (segment + 1)))
  // and on, disjoint for any lengths (a long sequence has one more segment than it has whole
  // ones at most), and fewer than `slots`.
  int segment;
  long slots;
  // Workspace, byte offsets.
  size_t off_states;           // [slot][Hv] states: before each segment, backward behind it
  size_t off_decay;            // [slot][Hv] float: the segment's whole decay
  size_t off_dots, off_dotk;   // backward: [linear_parts][Hv][tokens] parts of dg by rows (LinPass::dot)
  size_t off_inner;            // backward: [ceil(tokens / linear_chunk)][Hv][linear_parts] states before
                               // the chunks inside a segment, by waves
  size_t off_dgsum;            // backward: [sequences + chunk_slots][Hv] sums of dg over a chunk
  long chunk_slots;            // slots as above with a chunk as the segment
  size_t off_dq, off_dk;       // backward, Hv > Hk: [tokens][Hv][dk] float
  size_t total;
  // saved (training): [slot][Hv] states before each segment, [sequences][Hv] states before
  // sequences of one segment
  size_t off_first;
  size_t saved_total;
};

namespace s4 {

constexpr int kLinChunk = 64;    // tokens a chunk
constexpr int kDotParts = 16;    // waves that share the columns of a head, at most

// Tokens a chunk of a pass with dx columns, of tensors whose elements are `parts` bf16 parts: 32 where
// 64 do not fit into LDS.
constexpr int linear_chunk(int dx, int parts) { return dx > 128 && parts > 1 ? 32 : kLinChunk; }
// Rows of a state that a wave of a pass with dx columns holds, 16 columns of each.
constexpr int linear_rows(int dx) { return dx <= 64 ? 64 : dx <= 128 ? 128 : 256; }
constexpr int linear_type_parts(int dtype) { return dtype == S4DPLR_BF16 ? 1 : dtype == S4DPLR_F16 ? 2 : 3; }
constexpr long linear_slots(long tokens, int sequences, int segment) {
  const long most = tokens / (segment + 1);
  return most == 0 ? 0 : tokens / segment + (sequences < most ? sequences : most);
}

// Longest sequence that is taken token by token.  Token by token against by chunks, 16 heads of 128
// x 128 (us): bf16, 128 sequences, 4 tokens 64.2 against 66.6, 6 tokens 80.4 against 60.0; 16
// sequences, 4 tokens 12.8 against 12.9, 6 tokens 15.3 against 12.7; one, 6 tokens 10.0 against 10.7.  fp16 (two parts an element):
// 128 sequences, 8 tokens 94 against 108; 16 sequences, 6 tokens 15.9 against 15.3; one, 8 tokens
// 12.6 against 12.9.  fp32 (three parts): 128 sequences, 24 tokens 215 against 216; 16 sequences, 16
// tokens 29.1 against 29.8; one, 8 tokens 11.2 against 14.5, 16 tokens 18.6 against 14.4.
inline int lin_step_limit(const s4dplr_linear_attention_plan* p) {
  if (p->dtype == S4DPLR_BF16) return 5;
  if (p->dtype == S4DPLR_F16) return 6;
  return (long)p->sequences * p->Hv > 128 ? 16 : 10;
}

struct LinRows {
  long start, len;
  constexpr long slot(int s, int segment) const {
    const long before = start / (segment + 1);
    return start / segment + (s < before ? s : before);
  }
  constexpr int segments(int segment) const { return (int)((len + segment - 1) / segment); }
};

// One pass of the recurrence
//   out_t = read (decay to t) S^T x_t + pair sum_{j <= t} (decay from j to t) (x_t . y_j) w_j,
//   S <- (decay) S + update sum_j (decay from j) y_j w_j^T
// over all sequences, forwards or (rev) from their ends.  The forward pass and the three
// gradients are this pass with their tensors in other places.
struct LinPass {
  const void *x, *y, *w;
  long ldx, ldy, ldw;             // elements from one row to the next
  int gx, gy, gw;                 // value heads that share a head of x, y, w
  int dx, dw;
  void* out;                      // [tokens][Hv][dw]
  int out_f32;                    // out is float, not the tensors' type
  const float* g;                 // NULL: no decay
  long ldg;                       // Hv, or 0: one decay a head
  const int* offsets;
  const float* first;             // states before the first rows, NULL: zeros
  const float* before;            // [slot] states before the segments
  float* last;                    // states behind the last rows, may be NULL
  float* copy;                    // [sequences] states before sequences of one segment, may be NULL
  long rs, cs;                    // a state's element (row of dx, column of dw) is at rs row + cs column
  float read, pair, update;
  int rev;
  // The decays' gradient (dot not NULL): sums over the columns of `dot` times what out has from the
  // state before the chunk, read (decay to t) S^T x_t, by waves: [part][Hv][tokens].  Forwards, the
  // states before the chunks inside a segment go to `inner`.  In reverse, they are read from there, those
  // before segments from inner_slots and inner_first, and their inner products with the state behind the
  // chunk, times the chunk's decay, take the place of the last row's sum, which dg has no use for.
  const void* dot;
  long lddot;
  int gdot;
  float* dot_out;
  float* inner;                   // of the chunk that begins in row `token`: token / chunk
  const float *inner_first, *inner_slots;
  float* states;                  // the sums' pass: [slot] what each segment adds
  float* decay;                   // [slot][Hv]
  int sequences, each, Hv, dk, dv, segment;
  long tokens, slots;
  int step_tokens;                // sequences of at most so many rows are not this pass's
};

struct LinStep {
  const void *q, *k, *v;
  long ldq, ldk, ldv;
  const float* g;
  long ldg;
  const int* offsets;
  float scale;
  const float* state;
  void* o;
  float* state_out;
  int sequences, each, Hk, Hv, dk, dv, step_tokens;
  long tokens;
};

hipError_t launch_linear_steps(const LinStep& a, int dtype, hipStream_t s);
// What the segments add to the states, then (scan) the states before them.
hipError_t launch_linear_sums(const LinPass& a, int dtype, hipStream_t s);
hipError_t launch_linear_pass(const LinPass& a, int dtype, hipStream_t s);
// Each out [tokens][Hk][d] = the sums over each group of heads of part [tokens][Hv][d], in the
// sequences' rows.
struct LinGroups {
  const float* part[2];
  void* out[2];                   // may be NULL
  const int* offsets;
  int sequences, Hk, Hv, d;
  long tokens;
};
hipError_t launch_linear_groups(const LinGroups& a, int dtype, hipStream_t s);
// dg from the passes' sums by rows and the pairs inside the chunks; dg is [tokens][Hv] or (ldg == 0) [Hv].
struct LinGates {
  const void *q, *k, *v, *dout;
  long ldq, ldk, ldv, lddout;
  int dtype, group, dk, dv;
  float scale;
  const float *dots, *dotk;
  int parts;
  float *dg, *sums;
  const float* g;
  long ldg;
  const int* offsets;
  int sequences, each, Hv, segment;   // segment: the chunk
  long tokens, slots;
};
hipError_t launch_linear_gates(const LinGates& a, hipStream_t s);
// Waves that share the columns of a pass with these sizes.
int linear_parts(int dx, int dw, int dtype);

}  // namespace s4
