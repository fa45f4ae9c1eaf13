// Host side of the token-major operators: argument validation, the delta rule's
// plan and buffer layout, and the order of kernel launches.
#include <hip/hip_runtime_api.h>

#include <cmath>
#include <cstdint>
#include <new>

#include "delta.h"
#include "internal.h"
#include "norm.h"
#include "s4dplr.h"

namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool valid_dtype(int d) { return d == S4DPLR_F32 || d == S4DPLR_BF16 || d == S4DPLR_F16; }
size_t elem(int dtype) { return dtype == S4DPLR_F32 ? 4 : 2; }

// A buffer of the call: address, bytes, bytes its address is a multiple of.
struct Buf {
  const void* p;
  size_t n, align;
};

bool overlaps(const Buf& a, const Buf& b) {
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

s4dplr_status done(hipError_t e) { return e == hipSuccess ? S4DPLR_OK : s4::hip_failure(e); }

s4dplr_status norm_shape(long outer, long D, long inner) {
  if (outer < 0 || D < 1 || D > s4::kNormMaxD || inner < 1) return S4DPLR_ERR_SHAPE;
  const long most = inner == 1 ? 1L << 31 : 1L << 28;   // 512 threads per 64 vectors
  if (inner >= most || outer >= most || outer * inner >= most) return S4DPLR_ERR_SHAPE;
  return S4DPLR_OK;
}

size_t norm_part_bytes(long outer, long D, long inner) {
  return align_up(sizeof(float) * 2 * (size_t)s4::norm_parts(outer, D, inner) * (size_t)D);
}

}  // namespace

extern "C" {

s4dplr_status s4dplr_layer_norm_fwd(const void* x, const float* gamma, const float* beta, void* y,
                                    float* mean, float* rstd, long outer, long D, long inner,
                                    float eps, int dtype, hipStream_t stream) {
  if (!valid_dtype(dtype)) return S4DPLR_ERR_UNSUPPORTED;
  if (s4dplr_status st = norm_shape(outer, D, inner)) return st;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return S4DPLR_ERR_SHAPE;
  if (outer == 0) return S4DPLR_OK;
  if (!x || !y) return S4DPLR_ERR_NULL;
  const size_t es = elem(dtype), xb = es * (size_t)outer * D * inner;
  const size_t sb = sizeof(float) * (size_t)outer * inner, gb = sizeof(float) * (size_t)D;
  const Buf in[] = {{x, xb, es}, {gamma, gb, 4}, {beta, gb, 4}};
  const Buf out[] = {{y, xb, es}, {mean, sb, 4}, {rstd, sb, 4}};
  if (s4dplr_status st = check_buffers(in, out, 0, 0)) return st;
  s4::NormArgs a = {};
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.outer = outer;
  a.D = D;
  a.inner = inner;
  a.eps = eps;
  return done(s4::launch_norm_fwd(a, dtype, stream));
}

s4dplr_status s4dplr_layer_norm_workspace_bytes(long outer, long D, long inner, size_t* bytes) {
  if (!bytes) return S4DPLR_ERR_NULL;
  if (s4dplr_status st = norm_shape(outer, D, inner)) return st;
  *bytes = norm_part_bytes(outer, D, inner);
  return S4DPLR_OK;
}

s4dplr_status s4dplr_layer_norm_bwd(const void* x, const float* gamma, const float* mean,
                                    const float* rstd, const void* dy, void* dx, float* dgamma,
                                    float* dbeta, long outer, long D, long inner, int dtype,
                                    void* ws, hipStream_t stream) {
  if (!valid_dtype(dtype)) return S4DPLR_ERR_UNSUPPORTED;
  if (s4dplr_status st = norm_shape(outer, D, inner)) return st;
  if (outer > 0 && (!x || !mean || !rstd || !dy)) return S4DPLR_ERR_NULL;
  if (!ws) return S4DPLR_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(ws) % kAlign) return S4DPLR_ERR_WORKSPACE;
  const size_t es = elem(dtype), xb = es * (size_t)outer * D * inner;
  const size_t sb = sizeof(float) * (size_t)outer * inner, gb = sizeof(float) * (size_t)D;
  const Buf in[] = {{x, xb, es}, {gamma, gb, 4}, {mean, sb, 4}, {rstd, sb, 4}, {dy, xb, es}};
  const Buf out[] = {{dx, xb, es}, {dgamma, gb, 4}, {dbeta, gb, 4},
                     {ws, norm_part_bytes(outer, D, inner), kAlign}};
  if (s4dplr_status st = check_buffers(in, out, -1, -1)) return st;
  s4::NormArgs a = {};
  a.x = x;
  a.gamma = gamma;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dy = dy;
  a.dx = dx;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.part = static_cast<float*>(ws);
  a.outer = outer;
  a.D = D;
  a.inner = inner;
  if (!dgamma && !dbeta && (!dx || outer == 0)) return S4DPLR_OK;
  return done(s4::launch_norm_bwd(a, dtype, stream));
}

s4dplr_status s4dplr_delta_plan_create(s4dplr_delta_plan** out, int sequences, long tokens,
                                       int Hk, int Hv, int dk, int dv, int dtype,
                                       unsigned flags) {
  if (!out) return S4DPLR_ERR_NULL;
  *out = nullptr;
  if (!valid_dtype(dtype) || (flags & ~S4DPLR_DELTA_TRAINING)) return S4DPLR_ERR_UNSUPPORTED;
  if (sequences < 1 || tokens < 0 || tokens >= (1L << 31)) return S4DPLR_ERR_SHAPE;
  if (dk < 1 || dk > 256 || dv < 1 || dv > 256) return S4DPLR_ERR_SHAPE;
  if (Hk < 1 || Hv < 1 || Hv > 65535 || Hv % Hk) return S4DPLR_ERR_SHAPE;
  // a launch counts its threads in 32 bits: slices of a head x 512, chunks x 4 x 256
  if ((long)sequences * Hv > (1L << 18) || tokens * Hv >= (1L << 31) ||
      tokens / s4::kChunk + sequences >= (1L << 22) - 8)
    return S4DPLR_ERR_SHAPE;
  s4dplr_delta_plan* p = new (std::nothrow) s4dplr_delta_plan();
  if (!p) return S4DPLR_ERR_SHAPE;
  p->sequences = sequences;
  p->tokens = tokens;
  p->each = (int)(tokens / sequences);
  p->Hk = Hk;
  p->Hv = Hv;
  p->dk = dk;
  p->dv = dv;
  p->dtype = dtype;
  p->training = (flags & S4DPLR_DELTA_TRAINING) != 0;
  p->dkp = dk <= 64 ? 64 : dk <= 128 ? 128 : 256;
  p->parts = dtype == S4DPLR_BF16 ? 1 : dtype == S4DPLR_F16 ? 2 : 3;
  p->slots = s4::chunk_slots(p);
  const size_t ks = (size_t)p->slots * Hk, vs = (size_t)p->slots * Hv;
  const size_t kb = (size_t)p->parts * (p->dkp / 8) * s4::kFrag;   // 64 x dkp, all parts
  size_t off = 0;
  auto take = [&off](size_t n) {
    const size_t at = off;
    off = align_up(off + n);
    return at;
  };
  p->off_k = take(ks * kb);
  p->off_q = take(ks * kb);
  p->off_kt = take(ks * kb);
  p->off_x = take(vs * 3 * 8 * s4::kFrag);
  p->off_p = take(vs * 3 * 8 * s4::kFrag);
  p->off_vec = take(vs * sizeof(s4::DeltaVec));
  if (p->training) {
    p->off_qt = take(ks * kb);
    p->off_dv = take(vs * s4::kChunk * dv * sizeof(float));
    p->off_ds = take(vs * dk * dv * sizeof(float));
    p->off_gates = take(dk > 64 ? (size_t)((dk + 63) / 64) * 2 * tokens * Hv * sizeof(float) : 0);
  }
  p->total = off > 0 ? off : kAlign;   // never none: a caller's pointer to it is not NULL
  off = 0;
  p->off_n = take(vs * s4::kChunk * dv * sizeof(float));
  p->off_s = take(vs * dk * dv * sizeof(float));
  p->saved_total = p->training ? (off > 0 ? off : kAlign) : 0;
  *out = p;
  return S4DPLR_OK;
}

void s4dplr_delta_plan_destroy(s4dplr_delta_plan* p) { delete p; }

s4dplr_status s4dplr_delta_plan_bytes(const s4dplr_delta_plan* p, size_t* workspace,
                                      size_t* saved) {
  if (!p || !workspace) return S4DPLR_ERR_NULL;
  *workspace = p->total;
  if (saved) *saved = p->saved_total;
  return S4DPLR_OK;
}

// What the two passes check alike, and the shared part of the arguments.
static s4dplr_status delta_inputs(const s4dplr_delta_plan* p, const void* q, long ldq,
                                  const void* k, long ldk, const void* v, long ldv,
                                  const float* g, const float* beta, const int* offsets,
                                  float scale, const void* ws, s4::DeltaArgs* a, Buf (&in)[6]) {
  if (!p) return S4DPLR_ERR_NULL;
  if (p->tokens > 0 && (!q || !k || !v || !g || !beta)) return S4DPLR_ERR_NULL;
  if (!ws) return S4DPLR_ERR_NULL;
  const long wk = (long)p->Hk * p->dk, wv = (long)p->Hv * p->dv;
  constexpr long most = 1L << 24;   // offsets inside a chunk fit 32 bits
  if (ldq < wk || ldk < wk || ldv < wv || ldq >= most || ldk >= most || ldv >= most)
    return S4DPLR_ERR_SHAPE;
  if (!offsets && p->tokens % p->sequences) return S4DPLR_ERR_SHAPE;
  if (reinterpret_cast<uintptr_t>(ws) % kAlign) return S4DPLR_ERR_WORKSPACE;
  const size_t es = elem(p->dtype);
  auto span = [&](long ld, long width) {
    return p->tokens ? es * ((size_t)(p->tokens - 1) * ld + width) : 0;
  };
  const size_t gb = sizeof(float) * (size_t)p->tokens * p->Hv;
  in[0] = {q, span(ldq, wk), es};
  in[1] = {k, span(ldk, wk), es};
  in[2] = {v, span(ldv, wv), es};
  in[3] = {g, gb, 4};
  in[4] = {beta, gb, 4};
  in[5] = {offsets, sizeof(int) * ((size_t)p->sequences + 1), 4};
  a->q = q;
  a->k = k;
  a->v = v;
  a->ldq = ldq;
  a->ldk = ldk;
  a->ldv = ldv;
  a->g = g;
  a->beta = beta;
  a->offsets = offsets;
  a->scale = scale;
  a->ws = static_cast<unsigned char*>(const_cast<void*>(ws));
  a->step_tokens = -1;
  a->least = 1;
  return S4DPLR_OK;
}

s4dplr_status s4dplr_delta_fwd(const s4dplr_delta_plan* p, const void* q, long ldq, const void* k,
                               long ldk, const void* v, long ldv, const float* g,
                               const float* beta, const int* offsets, float scale,
                               const float* state, void* o, float* state_out, void* saved,
                               void* ws, hipStream_t stream) {
  s4::DeltaArgs a = {};
  Buf shared[6];
  if (s4dplr_status st =
          delta_inputs(p, q, ldq, k, ldk, v, ldv, g, beta, offsets, scale, ws, &a, shared))
    return st;
  if (p->tokens > 0 && !o) return S4DPLR_ERR_NULL;
  if (saved && !p->training) return S4DPLR_ERR_UNSUPPORTED;
  if (saved && reinterpret_cast<uintptr_t>(saved) % kAlign) return S4DPLR_ERR_WORKSPACE;
  const size_t es = elem(p->dtype);
  const size_t sb = sizeof(float) * (size_t)p->sequences * p->Hv * p->dk * p->dv;
  const Buf in[] = {{state, sb, 4}, shared[0], shared[1], shared[2],
                    shared[3],      shared[4], shared[5]};
  const Buf out[] = {{state_out, sb, 4},
                     {o, es * (size_t)p->tokens * p->Hv * p->dv, es},
                     {saved, p->saved_total, kAlign},
                     {ws, p->total, kAlign}};
  if (s4dplr_status st = check_buffers(in, out, 0, 0)) return st;
  a.state = state;
  a.o = o;
  a.state_out = state_out;
  a.saved = static_cast<unsigned char*>(saved);
  bool steps = false, chunks = true;
  if (!saved) {
    const long limit = s4::step_limit(p);
    chunks = (offsets ? p->tokens : p->each) > limit;
    steps = !chunks || (offsets && s4::packed_steps(p));
    if (steps) {
      a.step_tokens = (int)limit;
      a.least = (int)limit + 1;
    }
  }
  hipError_t e = hipSuccess;
  if (chunks) {
    if ((e = s4::launch_delta_prep(p, a, false, stream)) != hipSuccess) return done(e);
    if ((e = s4::launch_delta_scan(p, a, stream)) != hipSuccess) return done(e);
  }
  if (steps) e = s4::launch_delta_steps(p, a, stream);
  return done(e);
}

s4dplr_status s4dplr_delta_bwd(const s4dplr_delta_plan* p, const void* q, long ldq, const void* k,
                               long ldk, const void* v, long ldv, const float* g,
                               const float* beta, const int* offsets, float scale,
                               const void* saved, const void* dout, const float* dstate_out,
                               void* dq, void* dk, void* dv, float* dg, float* dbeta,
                               float* dstate, void* ws, hipStream_t stream) {
  s4::DeltaArgs a = {};
  Buf shared[6];
  if (s4dplr_status st =
          delta_inputs(p, q, ldq, k, ldk, v, ldv, g, beta, offsets, scale, ws, &a, shared))
    return st;
  if (!saved || (p->tokens > 0 && !dout)) return S4DPLR_ERR_NULL;
  if (!p->training) return S4DPLR_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(saved) % kAlign) return S4DPLR_ERR_WORKSPACE;
  const size_t es = elem(p->dtype);
  const size_t sb = sizeof(float) * (size_t)p->sequences * p->Hv * p->dk * p->dv;
  const size_t qb = es * (size_t)p->tokens * p->Hk * p->dk;
  const size_t vb = es * (size_t)p->tokens * p->Hv * p->dv;
  const size_t gb = sizeof(float) * (size_t)p->tokens * p->Hv;
  const Buf in[] = {{dstate_out, sb, 4}, shared[0], shared[1], shared[2],      shared[3],
                    shared[4],           shared[5], {dout, vb, es}, {saved, p->saved_total, kAlign}};
  const Buf out[] = {{dstate, sb, 4}, {dq, qb, es}, {dk, qb, es}, {dv, vb, es},
                     {dg, gb, 4},     {dbeta, gb, 4}, {ws, p->total, kAlign}};
  if (s4dplr_status st = check_buffers(in, out, 0, 0)) return st;
  a.dout = dout;
  a.dstate_out = dstate_out;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.dg = dg;
  a.dbeta = dbeta;
  a.dstate = dstate;
  a.saved = static_cast<unsigned char*>(const_cast<void*>(saved));
  hipError_t e;
  if ((e = s4::launch_delta_prep(p, a, true, stream)) != hipSuccess) return done(e);
  if ((e = s4::launch_delta_scan_bwd(p, a, stream)) != hipSuccess) return done(e);
  if (dq || dk || dg || dbeta) e = s4::launch_delta_grads(p, a, stream);
  return done(e);
}

}  // extern "C"
