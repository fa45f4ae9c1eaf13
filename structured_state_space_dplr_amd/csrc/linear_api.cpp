// Host side of linear attention: the plan and its buffers' layout, argument validation, and
// the order of kernel launches.
#include <hip/hip_runtime_api.h>

#include <new>

#include "buffers.h"
#include "linear.h"

namespace {

using namespace s4;

typedef s4dplr_linear_attention_plan Plan;

// Tokens of a segment: two blocks for each of the 256 CUs where there is enough work, a block per CU
// where there is less, and shorter segments, down to one chunk, where a call is bound by the
// dependent steps of a block.  Against that, each segment's state is written, read and written
// again, and read.  Forward, 16 heads of 128 x 128 in bf16 (us; chunks times heads, then the
// chunks of a segment with the time): 256: 1 29.2, 2 31.3, 4 42.8; 512: 1 44.1, 2 37.9, 4 46.1;
// 1024: 2 59.1, 4 52.9, 8 72.6; 2048: 2 104, 4 80.3, 8 80.1; 4096: 4 151, 8 125, 16 135; 16384 in 64
// sequences: 8 452, 16 (whole sequences) 329.  Training step of 4096: 4 747, 8 687, 16 938; of 2048: 4
// 374, 8 389, 16 592.
int segment_of(const Plan& p) {
  const long work = (p.tokens + kLinChunk - 1) / kLinChunk * p.Hv * ((p.dv + 127) / 128);
  const long n = (work + 511) / 512;
  return (int)(work <= 384 ? 1 : work <= 768 ? 2 : n < 4 ? 4 : n) * kLinChunk;
}

struct Inputs {
  const void *q, *k, *v;
  long ldq, ldk, ldv;
  const float* g;
  int g_fixed;
  const int* offsets;
  float scale;
};

s4dplr_status check_inputs(const Plan* p, const Inputs& a, const void* ws, Buf (&in)[5]) {
  if (!p) return S4DPLR_ERR_NULL;
  if (p->tokens > 0 && (!a.q || !a.k || !a.v)) return S4DPLR_ERR_NULL;
  if (!ws) return S4DPLR_ERR_NULL;
  const long wk = (long)p->Hk * p->dk, wv = (long)p->Hv * p->dv;
  constexpr long most = 1L << 24;
  if (a.ldq < wk || a.ldk < wk || a.ldv < wv || a.ldq >= most || a.ldk >= most || a.ldv >= most)
    return S4DPLR_ERR_SHAPE;
  if (!a.offsets && p->tokens % p->sequences) return S4DPLR_ERR_SHAPE;
  if (reinterpret_cast<uintptr_t>(ws) % kAlign) return S4DPLR_ERR_WORKSPACE;
  const size_t es = elem(p->dtype);
  auto span = [&](long ld, long width) {
    return p->tokens ? es * ((size_t)(p->tokens - 1) * ld + width) : 0;
  };
  in[0] = {a.q, span(a.ldq, wk), es};
  in[1] = {a.k, span(a.ldk, wk), es};
  in[2] = {a.v, span(a.ldv, wv), es};
  in[3] = {a.g, sizeof(float) * (a.g_fixed ? 1 : (size_t)p->tokens) * p->Hv, 4};
  in[4] = {a.offsets, sizeof(int) * ((size_t)p->sequences + 1), 4};
  return S4DPLR_OK;
}

// What the passes of a call have alike.
LinPass base(const Plan* p, const Inputs& a) {
  LinPass l = {};
  l.gx = l.gy = l.gw = l.gdot = 1;
  l.g = a.g;
  l.ldg = a.g_fixed ? 0 : p->Hv;
  l.offsets = a.offsets;
  l.sequences = p->sequences;
  l.each = p->each;
  l.Hv = p->Hv;
  l.dk = p->dk;
  l.dv = p->dv;
  l.segment = p->segment;
  l.tokens = p->tokens;
  l.slots = p->slots;
  l.step_tokens = -1;
  l.read = l.pair = l.update = 1.f;
  return l;
}

// The state as it lies in memory, rows of dk, or turned.
void natural(LinPass& l) {
  l.dx = l.dk;
  l.dw = l.dv;
  l.rs = l.dv;
  l.cs = 1;
}
void turned(LinPass& l) {
  l.dx = l.dv;
  l.dw = l.dk;
  l.rs = 1;
  l.cs = l.dv;
}

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<unsigned char*>(ws) + off);
}

}  // namespace

extern "C" {

s4dplr_status s4dplr_linear_attention_plan_create(s4dplr_linear_attention_plan** out, int sequences,
                                                  long tokens, int Hk, int Hv, int dk, int dv,
                                                  int dtype, unsigned flags) {
  if (!out) return S4DPLR_ERR_NULL;
  *out = nullptr;
  if (!valid_dtype(dtype) || (flags & ~S4DPLR_LINEAR_ATTENTION_TRAINING)) return S4DPLR_ERR_UNSUPPORTED;
  if (sequences < 1 || tokens < 0 || tokens >= (1L << 31)) return S4DPLR_ERR_SHAPE;
  if (dk < 1 || dk > 256 || dv < 1 || dv > 256) return S4DPLR_ERR_SHAPE;
  if (Hk < 1 || Hv < 1 || Hv > 65535 || Hv % Hk) return S4DPLR_ERR_SHAPE;
  // a launch counts its threads in 32 bits
  if ((long)sequences * Hv > (1L << 18) || tokens * Hv >= (1L << 31)) return S4DPLR_ERR_SHAPE;
  Plan* p = new (std::nothrow) Plan();
  if (!p) return S4DPLR_ERR_SHAPE;
  p->sequences = sequences;
  p->tokens = tokens;
  p->each = (int)(tokens / sequences);
  p->Hk = Hk;
  p->Hv = Hv;
  p->dk = dk;
  p->dv = dv;
  p->dtype = dtype;
  p->training = (flags & S4DPLR_LINEAR_ATTENTION_TRAINING) != 0;
  p->segment = segment_of(*p);
  p->slots = linear_slots(tokens, sequences, p->segment);
  const size_t state = sizeof(float) * (size_t)Hv * dk * dv;
  size_t off = 0;
  auto take = [&off](size_t n) {
    const size_t here = off;
    off = align_up(off + n);
    return here;
  };
  p->off_states = take(p->slots * state);
  p->off_decay = take(sizeof(float) * p->slots * Hv);
  if (p->training) {
    const int chunk = linear_chunk(dv, linear_type_parts(dtype));
    const size_t parts = (size_t)Hv * linear_parts(dv, dk, dtype), dots = sizeof(float) * parts * tokens;
    p->off_dots = take(dots);
    p->off_dotk = take(dots);
    // none where a segment is one chunk
    const long inside = p->segment > chunk && tokens > chunk ? (tokens + chunk - 1) / chunk : 0;
    p->off_inner = take(sizeof(float) * parts * inside * linear_rows(dv) * 16);
    p->chunk_slots = linear_slots(tokens, sequences, chunk);
    p->off_dgsum = take(sizeof(float) * ((size_t)sequences + p->chunk_slots) * Hv);
    const size_t grads = Hv > Hk ? sizeof(float) * (size_t)tokens * Hv * dk : 0;
    p->off_dq = take(grads);
    p->off_dk = take(grads);
  }
  p->total = off > 0 ? off : kAlign;   // never none: a caller's pointer to it is not NULL
  off = 0;
  take(p->slots * state);
  p->off_first = take((size_t)sequences * state);
  p->saved_total = p->training ? (off > 0 ? off : kAlign) : 0;
  *out = p;
  return S4DPLR_OK;
}

void s4dplr_linear_attention_plan_destroy(s4dplr_linear_attention_plan* p) { delete p; }

s4dplr_status s4dplr_linear_attention_plan_bytes(const s4dplr_linear_attention_plan* p,
                                                 size_t* workspace, size_t* saved) {
  if (!p || !workspace) return S4DPLR_ERR_NULL;
  *workspace = p->total;
  if (saved) *saved = p->saved_total;
  return S4DPLR_OK;
}

s4dplr_status s4dplr_linear_attention_fwd(const s4dplr_linear_attention_plan* p, const void* q,
                                          long ldq, const void* k, long ldk, const void* v, long ldv,
                                          const float* g, int g_fixed, const int* offsets,
                                          float scale, const float* state, void* o,
                                          float* state_out, void* saved, void* ws,
                                          hipStream_t stream) {
  const Inputs a = {q, k, v, ldq, ldk, ldv, g, g_fixed, offsets, scale};
  Buf shared[5];
  if (s4dplr_status st = check_inputs(p, a, ws, shared)) return st;
  if (p->tokens > 0 && !o) return S4DPLR_ERR_NULL;
  if (saved && !p->training) return S4DPLR_ERR_UNSUPPORTED;
  if (saved && reinterpret_cast<uintptr_t>(saved) % kAlign) return S4DPLR_ERR_WORKSPACE;
  const size_t es = elem(p->dtype);
  const size_t sb = sizeof(float) * (size_t)p->sequences * p->Hv * p->dk * p->dv;
  const Buf in[] = {{state, sb, 4}, shared[0], shared[1], shared[2], shared[3], shared[4]};
  const Buf out[] = {{state_out, sb, 4},
                     {o, es * (size_t)p->tokens * p->Hv * p->dv, es},
                     {saved, p->saved_total, kAlign},
                     {ws, p->total, kAlign}};
  if (s4dplr_status st = check_buffers(in, out, 0, 0)) return st;
  bool steps = false, chunks = true;
  const int limit = lin_step_limit(p);
  if (!saved) {
    // short sequences of a packed batch go token by token where sequences are short in the
    // mean: the lengths are known to the device only
    chunks = (offsets ? p->tokens : p->each) > limit;
    steps = !chunks || (offsets && p->tokens <= (long)limit * p->sequences);
  }
  hipError_t e = hipSuccess;
  if (chunks) {
    LinPass l = base(p, a);
    natural(l);
    l.x = q;
    l.y = k;
    l.w = v;
    l.ldx = ldq;
    l.ldy = ldk;
    l.ldw = ldv;
    l.gx = l.gy = p->Hv / p->Hk;
    l.read = l.pair = scale;
    l.first = state;
    l.states = at<float>(saved ? saved : ws, saved ? 0 : p->off_states);
    l.decay = at<float>(ws, p->off_decay);
    l.before = l.states;
    l.out = o;
    l.last = state_out;
    l.copy = saved ? at<float>(saved, p->off_first) : nullptr;
    l.step_tokens = steps ? limit : -1;
    if ((e = launch_linear_sums(l, p->dtype, stream)) != hipSuccess) return done(e);
    if ((e = launch_linear_pass(l, p->dtype, stream)) != hipSuccess) return done(e);
  }
  if (steps) {
    LinStep l = {};
    l.q = q;
    l.k = k;
    l.v = v;
    l.ldq = ldq;
    l.ldk = ldk;
    l.ldv = ldv;
    l.g = g;
    l.ldg = g_fixed ? 0 : p->Hv;
    l.offsets = offsets;
    l.scale = scale;
    l.state = state;
    l.o = o;
    l.state_out = state_out;
    l.sequences = p->sequences;
    l.each = p->each;
    l.Hk = p->Hk;
    l.Hv = p->Hv;
    l.dk = p->dk;
    l.dv = p->dv;
    l.step_tokens = limit;
    l.tokens = p->tokens;
    e = launch_linear_steps(l, p->dtype, stream);
  }
  return done(e);
}

s4dplr_status s4dplr_linear_attention_bwd(const s4dplr_linear_attention_plan* p, const void* q,
                                          long ldq, const void* k, long ldk, const void* v, long ldv,
                                          const float* g, int g_fixed, const int* offsets,
                                          float scale, const void* saved, const void* dout,
                                          const float* dstate_out, void* dq, void* dk, void* dv,
                                          float* dg, float* dstate, void* ws, hipStream_t stream) {
  const Inputs a = {q, k, v, ldq, ldk, ldv, g, g_fixed, offsets, scale};
  Buf shared[5];
  if (s4dplr_status st = check_inputs(p, a, ws, shared)) return st;
  if (!saved || (p->tokens > 0 && !dout) || (dg && !g)) return S4DPLR_ERR_NULL;
  if (!p->training) return S4DPLR_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(saved) % kAlign) return S4DPLR_ERR_WORKSPACE;
  const size_t es = elem(p->dtype);
  const size_t sb = sizeof(float) * (size_t)p->sequences * p->Hv * p->dk * p->dv;
  const size_t qb = es * (size_t)p->tokens * p->Hk * p->dk;
  const size_t vb = es * (size_t)p->tokens * p->Hv * p->dv;
  const Buf in[] = {{dstate_out, sb, 4}, shared[0], shared[1], shared[2],
                    shared[3],           shared[4], {dout, vb, es}, {saved, p->saved_total, kAlign}};
  const Buf out[] = {{dstate, sb, 4}, {dq, qb, es}, {dk, qb, es},
                     {dv, vb, es},    {dg, shared[3].n, 4}, {ws, p->total, kAlign}};
  if (s4dplr_status st = check_buffers(in, out, 0, 0)) return st;
  const bool grouped = p->Hv > p->Hk;
  const int group = p->Hv / p->Hk;
  const long ldo = (long)p->Hv * p->dv;
  const float* before = at<float>(const_cast<void*>(saved), 0);
  const float* first = at<float>(const_cast<void*>(saved), p->off_first);
  float *dots = at<float>(ws, p->off_dots), *dotk = at<float>(ws, p->off_dotk);
  float* inner = at<float>(ws, p->off_inner);
  hipError_t e = hipSuccess;
  // from the ends: the gradient of the states, for dk and dv
  LinPass z = base(p, a);
  z.rev = 1;
  z.pair = z.update = scale;
  z.first = dstate_out;
  z.states = at<float>(ws, p->off_states);
  z.decay = at<float>(ws, p->off_decay);
  z.before = z.states;
  LinPass zv = z;
  natural(zv);
  zv.x = k;
  zv.y = q;
  zv.w = dout;
  zv.ldx = ldk;
  zv.ldy = ldq;
  zv.ldw = ldo;
  zv.gx = zv.gy = group;
  zv.out = dv;
  zv.last = dstate;
  if (dk || dv || dg || dstate)
    if ((e = launch_linear_sums(zv, p->dtype, stream)) != hipSuccess) return done(e);
  if (dq || dg) {
    LinPass l = base(p, a);
    turned(l);
    l.x = dout;
    l.y = v;
    l.w = k;
    l.ldx = ldo;
    l.ldy = ldv;
    l.ldw = ldk;
    l.gw = group;
    l.read = l.pair = scale;
    l.first = first;
    l.before = before;
    l.out = grouped && dq ? at<void>(ws, p->off_dq) : dq;
    l.out_f32 = grouped && dq;
    if (dg) {
      l.dot = q;
      l.lddot = ldq;
      l.gdot = group;
      l.dot_out = dots;
      l.inner = inner;
    }
    if ((e = launch_linear_pass(l, p->dtype, stream)) != hipSuccess) return done(e);
  }
  if (dk || dg) {   // before dv's, which may write dstate over dstate_out
    LinPass l = z;
    turned(l);
    l.x = v;
    l.y = dout;
    l.w = q;
    l.ldx = ldv;
    l.ldy = ldo;
    l.ldw = ldq;
    l.gw = group;
    l.out = grouped && dk ? at<void>(ws, p->off_dk) : dk;
    l.out_f32 = grouped && dk;
    if (dg) {
      l.dot = k;
      l.lddot = ldk;
      l.gdot = group;
      l.dot_out = dotk;
      l.inner = inner;
      l.inner_first = first;
      l.inner_slots = before;
    }
    if ((e = launch_linear_pass(l, p->dtype, stream)) != hipSuccess) return done(e);
  }
  if (dv || dstate)
    if ((e = launch_linear_pass(zv, p->dtype, stream)) != hipSuccess) return done(e);
  if (grouped && (dq || dk)) {
    const LinGroups l = {{at<float>(ws, p->off_dq), at<float>(ws, p->off_dk)}, {dq, dk}, offsets,
                         p->sequences, p->Hk, p->Hv, p->dk, p->tokens};
    if ((e = launch_linear_groups(l, p->dtype, stream)) != hipSuccess) return done(e);
  }
  if (dg) {
    LinGates l = {};
    l.q = q;
    l.k = k;
    l.v = v;
    l.dout = dout;
    l.ldq = ldq;
    l.ldk = ldk;
    l.ldv = ldv;
    l.lddout = ldo;
    l.dtype = p->dtype;
    l.group = group;
    l.dk = p->dk;
    l.dv = p->dv;
    l.scale = scale;
    l.dots = dots;
    l.dotk = dotk;
    l.parts = linear_parts(p->dv, p->dk, p->dtype);
    l.dg = dg;
    l.sums = at<float>(ws, p->off_dgsum);
    l.g = g;
    l.ldg = g_fixed ? 0 : p->Hv;
    l.offsets = offsets;
    l.sequences = p->sequences;
    l.each = p->each;
    l.Hv = p->Hv;
    l.segment = linear_chunk(p->dv, linear_type_parts(p->dtype));
    l.tokens = p->tokens;
    l.slots = p->chunk_slots;
    e = launch_linear_gates(l, stream);
  }
  return done(e);
}

}  // extern "C"
