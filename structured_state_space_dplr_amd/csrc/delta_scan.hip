// Gated delta rule, chunked form, stage 2: the chunks of a sequence one after
// another.  A block of 4 waves carries DS columns of one head's dk x dv state S
// through them:
//   R = V - e . (K S),  N = X R,  U = beta . N,
//   O = scale e . (Q S) + (scale P) U,  S <- e_last S + K^T (d . U).
// S stays in fp32 accumulators (wave w: dk rows 16 (w + 4 i)); as an operand it
// goes through LDS as three bf16 parts, and so do R and d . U.  The row tile w of
// K, Q, X and P belongs to wave w alone, so those operands go straight from
// memory to registers, a chunk ahead.
#include "delta_device.h"

namespace s4 {

namespace {

constexpr int DS = 16;

}  // namespace

template <typename T, int PARTS, int OUTS, int DKP, bool SAVE>
__global__ __launch_bounds__(256) void delta_scan_kernel(const s4dplr_delta_plan p,
                                                         const DeltaArgs a) {
  constexpr int KS = DKP / 32, TPW = DKP / 64;
  __shared__ __attribute__((aligned(16))) __bf16 st[3][DS][DKP + 8];
  __shared__ __attribute__((aligned(16))) __bf16 rt[3][DS][kChunk + 8];
  __shared__ __attribute__((aligned(16))) __bf16 ut[OUTS][DS][kChunk + 8];
  __shared__ __attribute__((aligned(16))) __bf16 du[3][DS][kChunk + 8];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int sh, slice;
  if (!slice_of(p.sequences * p.Hv, (p.dv + DS - 1) / DS, &sh, &slice)) return;
  const int s = sh / p.Hv, h = sh % p.Hv, hk = h / (p.Hv / p.Hk);
  const Rows r = rows_of(a.offsets, p.tokens, p.sequences, s);
  if (r.len <= a.step_tokens) return;
  const int nc = r.chunks();
  const long slot0 = r.first(s);
  const int col = slice * DS + (lane & 15), r0 = 4 * (lane >> 4);
  const bool colon = col < p.dv;
  constexpr size_t kbytes = (size_t)PARTS * 4 * KS * kFrag;

  v4f S[TPW];
#pragma unroll
  for (int i = 0; i < TPW; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int d = 16 * (w + 4 * i) + r0 + e;
      S[i][e] = a.state && colon && d < p.dk
                    ? a.state[((size_t)sh * p.dk + d) * p.dv + col] : 0.f;
    }
  auto put_state = [&] {
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      v4bf t[3];
      split4<3>(S[i], t);
#pragma unroll
      for (int q = 0; q < 3; ++q)
        *reinterpret_cast<v4bf*>(&st[q][lane & 15][16 * (w + 4 * i) + r0]) = t[q];
    }
  };
  put_state();

  for (int c = 0; c < nc; ++c) {
    const long slot = slot0 + c, t0 = r.start + (long)c * kChunk;
    const int n = (int)(r.len - (long)c * kChunk < kChunk ? r.len - (long)c * kChunk : kChunk);
    const size_t kslot = (size_t)slot * p.Hk + hk, vslot = (size_t)slot * p.Hv + h;
    const unsigned char* kf = a.ws + p.off_k + kslot * kbytes;
    const unsigned char* qf = a.ws + p.off_q + kslot * kbytes;
    const unsigned char* ktf = a.ws + p.off_kt + kslot * kbytes;
    const unsigned char* xf = a.ws + p.off_x + vslot * (3 * 8 * kFrag);
    const unsigned char* pf = a.ws + p.off_p + vslot * (OUTS * 8 * kFrag);
    const DeltaVec* vec = reinterpret_cast<const DeltaVec*>(a.ws + p.off_vec) + vslot;
    const int i0 = 16 * w + r0;
    const v4f ev = *reinterpret_cast<const v4f*>(vec->e + i0);
    const v4f dv = *reinterpret_cast<const v4f*>(vec->d + i0);
    const v4f bv = *reinterpret_cast<const v4f*>(vec->beta + i0);
    const float el = vec->e[kChunk - 1];
    v4f vv;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      vv[e] = colon && i0 + e < n
                  ? to_f32(((const T*)a.v)[(t0 + i0 + e) * a.ldv + (size_t)h * p.dv + col]) : 0.f;
    if constexpr (SAVE) {
      float* so = reinterpret_cast<float*>(a.saved + p.off_s) + vslot * p.dk * p.dv;
#pragma unroll
      for (int i = 0; i < TPW; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int d = 16 * (w + 4 * i) + r0 + e;
          if (colon && d < p.dk) so[(size_t)d * p.dv + col] = S[i][e];
        }
    }
    __syncthreads();
    v4f ks_ = {0.f, 0.f, 0.f, 0.f}, qs = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      v8bf ka[PARTS], qa[PARTS], sb[3];
#pragma unroll
      for (int i = 0; i < PARTS; ++i) {
        ka[i] = load_frag(kf, (i * 4 + w) * KS + ks, lane);
        qa[i] = load_frag(qf, (i * 4 + w) * KS + ks, lane);
      }
#pragma unroll
      for (int i = 0; i < 3; ++i)
        sb[i] = *reinterpret_cast<const v8bf*>(&st[i][lane & 15][ks * 32 + (lane >> 4) * 8]);
      ks_ = mfma_parts<3>(ka, sb, ks_);
      qs = mfma_parts<3>(qa, sb, qs);
    }
    {
      v4bf t[3];
      split4<3>(vv - ev * ks_, t);
#pragma unroll
      for (int q = 0; q < 3; ++q) *reinterpret_cast<v4bf*>(&rt[q][lane & 15][i0]) = t[q];
    }
    __syncthreads();
    v4f N = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      if (ks <= w / 2) {
        v8bf xa[3], rb[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          xa[i] = load_frag(xf, (i * 4 + w) * 2 + ks, lane);
          rb[i] = *reinterpret_cast<const v8bf*>(&rt[i][lane & 15][ks * 32 + (lane >> 4) * 8]);
        }
        N = mfma_parts<3>(xa, rb, N);
      }
    if constexpr (SAVE) {
      float* no = reinterpret_cast<float*>(a.saved + p.off_n) + vslot * kChunk * p.dv;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (colon) no[(size_t)(i0 + e) * p.dv + col] = N[e];
    }
    {
      const v4f U = bv * N;
      v4bf t[3], u[OUTS];
      split4<3>(dv * U, t);
      split4<OUTS>(U, u);
#pragma unroll
      for (int q = 0; q < 3; ++q) *reinterpret_cast<v4bf*>(&du[q][lane & 15][i0]) = t[q];
#pragma unroll
      for (int q = 0; q < OUTS; ++q) *reinterpret_cast<v4bf*>(&ut[q][lane & 15][i0]) = u[q];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      S[i] *= el;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        v8bf ta[PARTS], ub[3];
#pragma unroll
        for (int q = 0; q < PARTS; ++q)
          ta[q] = load_frag(ktf, (q * (DKP / 16) + w + 4 * i) * 2 + ks, lane);
#pragma unroll
        for (int q = 0; q < 3; ++q)
          ub[q] = *reinterpret_cast<const v8bf*>(&du[q][lane & 15][ks * 32 + (lane >> 4) * 8]);
        S[i] = mfma_parts<3>(ta, ub, S[i]);
      }
    }
    put_state();
    v4f o = qs * (ev * a.scale);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      if (ks <= w / 2) {
        v8bf pa[OUTS], ub[OUTS];
#pragma unroll
        for (int q = 0; q < OUTS; ++q) {
          pa[q] = load_frag(pf, (q * 4 + w) * 2 + ks, lane);
          ub[q] = *reinterpret_cast<const v8bf*>(&ut[q][lane & 15][ks * 32 + (lane >> 4) * 8]);
        }
        o = mfma_parts<OUTS>(pa, ub, o);
      }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (colon && i0 + e < n)
        ((T*)a.o)[((size_t)(t0 + i0 + e) * p.Hv + h) * p.dv + col] = from_f32<T>(o[e]);
  }
  if (a.state_out)
#pragma unroll
    for (int i = 0; i < TPW; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = 16 * (w + 4 * i) + r0 + e;
        if (colon && d < p.dk) a.state_out[((size_t)sh * p.dk + d) * p.dv + col] = S[i][e];
      }
}

// The same backwards, for the gradient Z of the state behind a chunk (dS' in the
// formulas):
//   dU = (scale P)^T dO + d . (K Z),  dV = X^T (beta . dU),
//   Z <- e_last Z + Q^T (scale e . dO) - K^T (e . dV).
// dV (the gradient of v, and in fp32 for stage 3) and Z before its update are
// written out.
template <typename T, int PARTS, int OUTS, int DKP>
__global__ __launch_bounds__(256) void delta_scan_bwd_kernel(const s4dplr_delta_plan p,
                                                             const DeltaArgs a) {
  constexpr int KS = DKP / 32, TPW = DKP / 64;
  __shared__ __attribute__((aligned(16))) __bf16 st[3][DS][DKP + 8];
  __shared__ __attribute__((aligned(16))) __bf16 ot[PARTS][DS][kChunk + 8];   // dO
  __shared__ __attribute__((aligned(16))) __bf16 et[3][DS][kChunk + 8];       // scale e . dO
  __shared__ __attribute__((aligned(16))) __bf16 ut[3][DS][kChunk + 8];       // beta . dU
  __shared__ __attribute__((aligned(16))) __bf16 vt[3][DS][kChunk + 8];       // -e . dV
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int sh, slice;
  if (!slice_of(p.sequences * p.Hv, (p.dv + DS - 1) / DS, &sh, &slice)) return;
  const int s = sh / p.Hv, h = sh % p.Hv, hk = h / (p.Hv / p.Hk);
  const Rows r = rows_of(a.offsets, p.tokens, p.sequences, s);
  if (r.len <= a.step_tokens) return;
  const int nc = r.chunks();
  const long slot0 = r.first(s);
  const int col = slice * DS + (lane & 15), r0 = 4 * (lane >> 4);
  const bool colon = col < p.dv;
  constexpr size_t kbytes = (size_t)PARTS * 4 * KS * kFrag;

  v4f Z[TPW];
#pragma unroll
  for (int i = 0; i < TPW; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int d = 16 * (w + 4 * i) + r0 + e;
      Z[i][e] = a.dstate_out && colon && d < p.dk
                    ? a.dstate_out[((size_t)sh * p.dk + d) * p.dv + col] : 0.f;
    }
  auto put_state = [&] {
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      v4bf t[3];
      split4<3>(Z[i], t);
#pragma unroll
      for (int q = 0; q < 3; ++q)
        *reinterpret_cast<v4bf*>(&st[q][lane & 15][16 * (w + 4 * i) + r0]) = t[q];
    }
  };
  put_state();

  for (int c = nc - 1; c >= 0; --c) {
    const long slot = slot0 + c, t0 = r.start + (long)c * kChunk;
    const int n = (int)(r.len - (long)c * kChunk < kChunk ? r.len - (long)c * kChunk : kChunk);
    const size_t kslot = (size_t)slot * p.Hk + hk, vslot = (size_t)slot * p.Hv + h;
    const unsigned char* kf = a.ws + p.off_k + kslot * kbytes;
    const unsigned char* ktf = a.ws + p.off_kt + kslot * kbytes;
    const unsigned char* qtf = a.ws + p.off_qt + kslot * kbytes;
    const unsigned char* xf = a.ws + p.off_x + vslot * (3 * 8 * kFrag);
    const unsigned char* pf = a.ws + p.off_p + vslot * (OUTS * 8 * kFrag);
    const DeltaVec* vec = reinterpret_cast<const DeltaVec*>(a.ws + p.off_vec) + vslot;
    const int i0 = 16 * w + r0;
    const v4f ev = *reinterpret_cast<const v4f*>(vec->e + i0);
    const v4f dv = *reinterpret_cast<const v4f*>(vec->d + i0);
    const v4f bv = *reinterpret_cast<const v4f*>(vec->beta + i0);
    const float el = vec->e[kChunk - 1];
    v4f go;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      go[e] = colon && i0 + e < n
                  ? to_f32(((const T*)a.dout)[((size_t)(t0 + i0 + e) * p.Hv + h) * p.dv + col])
                  : 0.f;
    {
      v4bf t[PARTS], u[3];
      split4<PARTS>(go, t);
      split4<3>(go * (ev * a.scale), u);
#pragma unroll
      for (int q = 0; q < PARTS; ++q) *reinterpret_cast<v4bf*>(&ot[q][lane & 15][i0]) = t[q];
#pragma unroll
      for (int q = 0; q < 3; ++q) *reinterpret_cast<v4bf*>(&et[q][lane & 15][i0]) = u[q];
    }
    float* zo = reinterpret_cast<float*>(a.ws + p.off_ds) + vslot * p.dk * p.dv;
#pragma unroll
    for (int i = 0; i < TPW; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = 16 * (w + 4 * i) + r0 + e;
        if (colon && d < p.dk) zo[(size_t)d * p.dv + col] = Z[i][e];
      }
    __syncthreads();
    v4f kz = {0.f, 0.f, 0.f, 0.f}, g1 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      v8bf ka[PARTS], sb[3];
#pragma unroll
      for (int i = 0; i < PARTS; ++i) ka[i] = load_frag(kf, (i * 4 + w) * KS + ks, lane);
#pragma unroll
      for (int i = 0; i < 3; ++i)
        sb[i] = *reinterpret_cast<const v8bf*>(&st[i][lane & 15][ks * 32 + (lane >> 4) * 8]);
      kz = mfma_parts<3>(ka, sb, kz);
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      if (ks >= w / 2) {
        v8bf pa[OUTS], ob[PARTS];
#pragma unroll
        for (int q = 0; q < OUTS; ++q) pa[q] = load_frag(pf, (q * 4 + w) * 2 + ks, lane);
#pragma unroll
        for (int q = 0; q < PARTS; ++q)
          ob[q] = *reinterpret_cast<const v8bf*>(&ot[q][lane & 15][ks * 32 + (lane >> 4) * 8]);
        g1 = mfma_parts<3>(pa, ob, g1);
      }
    {
      v4bf t[3];
      split4<3>(bv * (g1 + dv * kz), t);
#pragma unroll
      for (int q = 0; q < 3; ++q) *reinterpret_cast<v4bf*>(&ut[q][lane & 15][i0]) = t[q];
    }
    __syncthreads();
    v4f dV = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      if (ks >= w / 2) {
        v8bf xa[3], ub[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          xa[i] = load_frag(xf, (i * 4 + w) * 2 + ks, lane);
          ub[i] = *reinterpret_cast<const v8bf*>(&ut[i][lane & 15][ks * 32 + (lane >> 4) * 8]);
        }
        dV = mfma_parts<3>(xa, ub, dV);
      }
    float* vo = reinterpret_cast<float*>(a.ws + p.off_dv) + vslot * kChunk * p.dv;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (colon) {
        vo[(size_t)(i0 + e) * p.dv + col] = dV[e];
        if (a.dv && i0 + e < n)
          ((T*)a.dv)[((size_t)(t0 + i0 + e) * p.Hv + h) * p.dv + col] = from_f32<T>(dV[e]);
      }
    {
      v4bf t[3];
      split4<3>(-(ev * dV), t);
#pragma unroll
      for (int q = 0; q < 3; ++q) *reinterpret_cast<v4bf*>(&vt[q][lane & 15][i0]) = t[q];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      Z[i] *= el;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        v8bf ta[PARTS], qa[PARTS], vb[3], eb[3];
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
          ta[q] = load_frag(ktf, (q * (DKP / 16) + w + 4 * i) * 2 + ks, lane);
          qa[q] = load_frag(qtf, (q * (DKP / 16) + w + 4 * i) * 2 + ks, lane);
        }
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          vb[q] = *reinterpret_cast<const v8bf*>(&vt[q][lane & 15][ks * 32 + (lane >> 4) * 8]);
          eb[q] = *reinterpret_cast<const v8bf*>(&et[q][lane & 15][ks * 32 + (lane >> 4) * 8]);
        }
        Z[i] = mfma_parts<3>(ta, vb, Z[i]);
        Z[i] = mfma_parts<3>(qa, eb, Z[i]);
      }
    }
    __syncthreads();   // ot and et are written again
    put_state();
  }
  if (a.dstate)
#pragma unroll
    for (int i = 0; i < TPW; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = 16 * (w + 4 * i) + r0 + e;
        if (colon && d < p.dk) a.dstate[((size_t)sh * p.dk + d) * p.dv + col] = Z[i][e];
      }
}

namespace {

unsigned slice_blocks(const s4dplr_delta_plan* p) {
  const unsigned heads = (unsigned)(p->sequences * p->Hv);
  return (heads + 7) / 8 * 8 * ((p->dv + DS - 1) / DS);
}

template <typename T, int PARTS, int OUTS>
hipError_t scan(const s4dplr_delta_plan* p, const DeltaArgs& a, bool bwd, hipStream_t s) {
  const unsigned grid = slice_blocks(p);
#define S4_GO(dkp)                                                                     \
  if (bwd)                                                                             \
    delta_scan_bwd_kernel<T, PARTS, OUTS, dkp><<<grid, 256, 0, s>>>(*p, a);            \
  else if (a.saved)                                                                    \
    delta_scan_kernel<T, PARTS, OUTS, dkp, true><<<grid, 256, 0, s>>>(*p, a);          \
  else                                                                                 \
    delta_scan_kernel<T, PARTS, OUTS, dkp, false><<<grid, 256, 0, s>>>(*p, a)
  if (p->dkp == 64) { S4_GO(64); }
  else if (p->dkp == 128) { S4_GO(128); }
  else { S4_GO(256); }
#undef S4_GO
  return hipGetLastError();
}

hipError_t scan_any(const s4dplr_delta_plan* p, const DeltaArgs& a, bool bwd, hipStream_t s) {
  if (p->dtype == S4DPLR_F32) return scan<float, 3, 3>(p, a, bwd, s);
  if (p->dtype == S4DPLR_BF16) return scan<bf16, 1, 2>(p, a, bwd, s);
  return scan<f16, 2, 2>(p, a, bwd, s);
}

}  // namespace

hipError_t launch_delta_scan(const s4dplr_delta_plan* p, const DeltaArgs& a, hipStream_t s) {
  return scan_any(p, a, false, s);
}
hipError_t launch_delta_scan_bwd(const s4dplr_delta_plan* p, const DeltaArgs& a, hipStream_t s) {
  return scan_any(p, a, true, s);
}

}  // namespace s4
