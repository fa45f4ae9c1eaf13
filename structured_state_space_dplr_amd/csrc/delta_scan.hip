// Gated delta rule, chunked form, stage 2: the chunks of a sequence one after
// another.  A block carries DS columns of one head's dk x dv state S through them:
//   R = V - e . (K S),  N = X R,  U = beta . N,
//   O = scale e . (Q S) + (scale P) U,  S <- e_last S + K^T (d . U).
//
// A step is a chain of small products with an exchange between waves after each,
// so its time is latency and instruction issue, not bandwidth.  Of the 8 waves, 0 - 3
// walk the chain: wave w owns a quarter of S's rows in fp32 accumulators.  The
// accumulator layout (lane: column l % 16, rows 4 (l / 16) ..) is a matrix operand's
// layout with its k index permuted, and K and Q are stored in that permutation, so S
// enters K S and Q S straight from registers as three bf16 parts; the waves' partial
// sums meet in LDS.  R and d . U pass through LDS as bf16 parts.  Waves 4 - 7 sum Q S
// and compute and store O beside the chain.  The row tiles of X, P and K^T belong to
// one wave each: those operands go from memory to registers, a chunk ahead.
#include "delta_device.h"

namespace s4 {

namespace {

constexpr int DS = 16;
constexpr int kLdT = kChunk + 8;   // bf16 from column to column of a chunk-long operand
constexpr int kLdF = kChunk + 4;   // fp32 likewise

// Who owns which rows of the state.  DKP = 128, 256: wave w has the k steps (32
// rows each) w KW .. + KW and multiplies all four row tiles of a chunk with them.
// DKP = 64: two waves hold the same k step and take two row tiles each.
template <int DKP>
struct Own {
  static constexpr int KS = DKP / 32, KW = KS > 4 ? KS / 4 : 1;
  static constexpr int WAVES = KS < 4 ? 2 : 4;        // partial sums of a product
  static constexpr int RT = KS < 4 ? 2 : 4;           // row tiles of a chunk per wave
  __device__ static int kw(int w) { return KS < 4 ? w >> 1 : w; }
  __device__ static int rt(int w) { return KS < 4 ? 2 * (w & 1) : 0; }
  __device__ static bool first(int w) { return KS < 4 ? (w & 1) == 0 : true; }
};

// What both scans start from.
struct Place {
  int sh, h, hk, nc, col, ccol, lr, lg;
  bool colon;
  Rows r;
  long slot0;
};
__device__ __forceinline__ bool place_of(const s4dplr_delta_plan& p, const DeltaArgs& a, int lane,
                                         Place* o) {
  int slice;
  if (!slice_of(p.sequences * p.Hv, (p.dv + DS - 1) / DS, &o->sh, &slice)) return false;
  const int s = o->sh / p.Hv;
  o->h = o->sh % p.Hv;
  o->hk = o->h / (p.Hv / p.Hk);
  o->r = rows_of(p, a.offsets, s);
  o->nc = o->r.chunks();
  o->slot0 = o->r.first(s);
  o->lr = lane & 15;
  o->lg = lane >> 4;
  o->col = slice * DS + o->lr;
  o->colon = o->col < p.dv;
  o->ccol = o->colon ? o->col : 0;
  return true;
}

// The wave's rows of a state [dk][dv] in fp32: tile t of k step k is rows 32 k + 16 t
// + 4 lg ..
template <int KW>
__device__ __forceinline__ void load_state(v4f (&S)[KW][2], const float* state, int k0,
                                           const s4dplr_delta_plan& p, const Place& at) {
#pragma unroll
  for (int i = 0; i < KW; ++i)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = 32 * (k0 + i) + 16 * t + 4 * at.lg + e;
        S[i][t][e] = state && at.colon && d < p.dk
                         ? state[((size_t)at.sh * p.dk + d) * p.dv + at.col] : 0.f;
      }
}
template <int KW>
__device__ __forceinline__ void store_state(const v4f (&S)[KW][2], float* state, int k0,
                                            const s4dplr_delta_plan& p, const Place& at) {
  if (!state || !at.colon) return;
#pragma unroll
  for (int i = 0; i < KW; ++i)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = 32 * (k0 + i) + 16 * t + 4 * at.lg + e;
        if (d < p.dk) state[((size_t)at.sh * p.dk + d) * p.dv + at.col] = S[i][t][e];
      }
}
// A chunk's state for stage 3 of the backward pass, [dv][dk]: `to` is the lane's column.
template <int KW>
__device__ __forceinline__ void keep_state(const v4f (&S)[KW][2], float* to, int k0, int dk, int lg) {
#pragma unroll
  for (int i = 0; i < KW; ++i)
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int d = 32 * (k0 + i) + 16 * t + 4 * lg;
      if (d + 4 <= dk) {
        __builtin_memcpy(to + d, &S[i][t], 16);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (d + e < dk) to[d + e] = S[i][t][e];
      }
    }
}
// The rows of a k step as an operand of three parts.
__device__ __forceinline__ void state_operand(const v4f (&S)[2], v8bf (&out)[3]) {
  float x[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[e] = S[0][e];
    x[4 + e] = S[1][e];
  }
  split8<3>(x, out);
}

template <int N>
__device__ __forceinline__ void put4(__bf16 (*to)[DS][kLdT], v4f x, int lr, int i0) {
  v4bf t[N];
  split4<N>(x, t);
#pragma unroll
  for (int q = 0; q < N; ++q) *reinterpret_cast<v4bf*>(&to[q][lr][i0]) = t[q];
}
template <int N>
__device__ __forceinline__ void get8(const __bf16 (*from)[DS][kLdT], v8bf (&x)[N], int lr, int k) {
#pragma unroll
  for (int q = 0; q < N; ++q) x[q] = *reinterpret_cast<const v8bf*>(&from[q][lr][k]);
}

}  // namespace

template <typename T, int PARTS, int OUTS, int DKP, bool SAVE>
__global__ __launch_bounds__(512) void delta_scan_kernel(const s4dplr_delta_plan p,
                                                         const DeltaArgs a) {
  using O = Own<DKP>;
  constexpr int KS = O::KS, KW = O::KW, RT = O::RT;
  __shared__ __attribute__((aligned(16))) float pk[O::WAVES][DS][kLdF];   // K S, by owner
  __shared__ __attribute__((aligned(16))) float pq[O::WAVES][DS][kLdF];   // Q S
  __shared__ __attribute__((aligned(16))) __bf16 rt[3][DS][kLdT];         // R
  __shared__ __attribute__((aligned(16))) __bf16 ut[OUTS][DS][kLdT];      // U
  __shared__ __attribute__((aligned(16))) __bf16 du[3][DS][kLdT];         // d . U
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Place at;
  if (!place_of(p, a, lane, &at) || at.r.len <= a.step_tokens) return;
  const int lr = at.lr, lg = at.lg, w = wave & 3, i0 = 16 * w + 4 * lg, nc = at.nc;
  constexpr size_t kbytes = (size_t)PARTS * 4 * KS * kFrag;
  const size_t k0 = ((size_t)at.slot0 * p.Hk + at.hk) * kbytes;
  const size_t v0 = (size_t)at.slot0 * p.Hv + at.h;
  const size_t kstep = (size_t)p.Hk * kbytes;
  const unsigned off = lane * 16;
  const DeltaVec* dp = reinterpret_cast<const DeltaVec*>(a.ws + p.off_vec) + v0;
  const v4f zero = {0.f, 0.f, 0.f, 0.f};

  if (wave < 4) {
    __builtin_amdgcn_s_setprio(1);
    const int kw = O::kw(w) * KW, rt0 = O::rt(w);
    v4f S[KW][2];
    load_state<KW>(S, a.state, kw, p, at);

    // Operands of one chunk, each set loaded right after its last use.
    v8bf ka[KW][RT][PARTS], qa[KW][RT][PARTS], xa[2][3], ta[KW][2][2][PARTS];
    v4f ev, dv, bv;
    float el;
    T vv[4];
    const size_t kq0 = k0 + (size_t)(rt0 * KS + kw) * kFrag;
    const unsigned char* kp = a.ws + p.off_k + kq0;
    const unsigned char* qp = a.ws + p.off_q + kq0;
    const unsigned char* tp = a.ws + p.off_kt + k0 + (size_t)kw * 4 * kFrag;
    const unsigned char* xp = a.ws + p.off_x + v0 * (3 * 8 * kFrag) + (size_t)w * 2 * kFrag;
    const T* vp = (const T*)a.v + at.r.start * a.ldv + (size_t)at.h * p.dv;
    float* np = SAVE ? reinterpret_cast<float*>(a.saved + p.off_n) + v0 * kChunk * p.dv +
                           (size_t)at.ccol * kChunk + i0 : nullptr;
    float* sp = SAVE ? reinterpret_cast<float*>(a.saved + p.off_s) + v0 * p.dk * p.dv +
                           (size_t)at.ccol * p.dk : nullptr;
    const unsigned ldv = (unsigned)a.ldv;
    unsigned voff[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) voff[e] = (unsigned)(i0 + e) * ldv + at.ccol;
    auto load_kq = [&](const unsigned char* from, v8bf (&to)[KW][RT][PARTS]) {
#pragma unroll
      for (int q = 0; q < PARTS; ++q)
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int i = 0; i < KW; ++i) to[i][t][q] = load_frag(from, (q * 4 + t) * KS + i, off);
    };
    auto load_x = [&] {
#pragma unroll
      for (int i = 0; i < 3; ++i) xa[0][i] = load_frag(xp, i * 8, off);
      if (w >= 2)
#pragma unroll
        for (int i = 0; i < 3; ++i) xa[1][i] = load_frag(xp, i * 8 + 1, off);
    };
    auto load_t = [&] {
#pragma unroll
      for (int q = 0; q < PARTS; ++q)
#pragma unroll
        for (int i = 0; i < KW; ++i)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
              ta[i][t][ks][q] = load_frag(tp, (q * (DKP / 16) + 2 * i + t) * 2 + ks, off);
    };
    // A partial chunk's rows behind the end read the sequence's last row: their
    // K, Q and beta are zero, so their values reach nothing.  (A load under a
    // condition would be waited for at once.)
    auto load_v = [&](int c) {
      const int n = (int)(at.r.len - (long)c * kChunk);
      if (n >= kChunk) {
#pragma unroll
        for (int e = 0; e < 4; ++e) vv[e] = vp[voff[e]];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          vv[e] = vp[(unsigned)(i0 + e < n ? i0 + e : n - 1) * ldv + at.ccol];
      }
    };
    auto load_d = [&] {
      ev = *reinterpret_cast<const v4f*>(dp->e + i0);
      dv = *reinterpret_cast<const v4f*>(dp->d + i0);
      bv = *reinterpret_cast<const v4f*>(dp->beta + i0);
      el = dp->e[kChunk - 1];
    };
    if (nc > 0) {
      load_kq(kp, ka);
      load_v(0);
      load_d();
      load_kq(qp, qa);
      load_x();
      load_t();
    }
    for (int c = 0; c < nc; ++c) {
      const bool more = c + 1 < nc;   // else the same operands once more
      if (more) {
        kp += kstep;
        qp += kstep;
        tp += kstep;
        xp += (size_t)p.Hv * (3 * 8 * kFrag);
        dp += p.Hv;
        vp += (size_t)kChunk * ldv;
      }
      v8bf sb[KW][3];
#pragma unroll
      for (int i = 0; i < KW; ++i) state_operand(S[i], sb[i]);
      {
        v4f x[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) x[t] = zero;
#pragma unroll
        for (int i = 0; i < KW; ++i)
#pragma unroll
          for (int t = 0; t < RT; ++t) x[t] = mfma_parts<3>(ka[i][t], sb[i], x[t]);
        if (SAVE && at.colon && O::first(w)) keep_state<KW>(S, sp, kw, p.dk, lg);
        if constexpr (SAVE) sp += (size_t)p.Hv * p.dk * p.dv;
#pragma unroll
        for (int t = 0; t < RT; ++t)
          *reinterpret_cast<v4f*>(&pk[O::kw(w)][lr][16 * (rt0 + t) + 4 * lg]) = x[t];
      }
      load_kq(kp, ka);
      __syncthreads();
      {
        v4f ks[O::WAVES];
#pragma unroll
        for (int i = 0; i < O::WAVES; ++i) ks[i] = *reinterpret_cast<const v4f*>(&pk[i][lr][i0]);
        // off the chain: Q S
        v4f x[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) x[t] = zero;
#pragma unroll
        for (int i = 0; i < KW; ++i)
#pragma unroll
          for (int t = 0; t < RT; ++t) x[t] = mfma_parts<3>(qa[i][t], sb[i], x[t]);
        v4f R;
#pragma unroll
        for (int e = 0; e < 4; ++e) R[e] = to_f32(vv[e]);
        v4f sum = ks[0] + ks[1];
        if constexpr (O::WAVES == 4) sum += ks[2] + ks[3];
        put4<3>(rt, R - ev * sum, lr, i0);
#pragma unroll
        for (int t = 0; t < RT; ++t)
          *reinterpret_cast<v4f*>(&pq[O::kw(w)][lr][16 * (rt0 + t) + 4 * lg]) = x[t];
      }
      load_v(c + more);
      __syncthreads();
      v4f N = zero, n1 = zero;
      {
        v8bf rb[3], rc[3];
        get8<3>(rt, rb, lr, lg * 8);
        if (w >= 2) {
          get8<3>(rt, rc, lr, 32 + lg * 8);
          n1 = mfma_parts<3>(xa[1], rc, n1);
        }
        N = mfma_parts<3>(xa[0], rb, N);
        N += n1;
      }
      {
        const v4f U = bv * N;
        put4<3>(du, dv * U, lr, i0);
        put4<OUTS>(ut, U, lr, i0);
      }
      load_kq(qp, qa);
      load_x();
      if constexpr (SAVE) {
        if (at.colon) *reinterpret_cast<v4f*>(np) = N;
        np += (size_t)p.Hv * kChunk * p.dv;
      }
      __syncthreads();
      v8bf ub[2][3];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) get8<3>(du, ub[ks], lr, ks * 32 + lg * 8);
#pragma unroll
      for (int i = 0; i < KW; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t) S[i][t] *= el;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int i = 0; i < KW; ++i)
#pragma unroll
          for (int t = 0; t < 2; ++t) S[i][t] = mfma_parts<3>(ta[i][t][ks], ub[ks], S[i][t]);
      load_d();
      load_t();
    }
    if (O::first(w)) store_state<KW>(S, a.state_out, kw, p, at);
  } else {
    v8bf pa[2][OUTS];
    v4f ev;
    const unsigned char* pp = a.ws + p.off_p + v0 * (OUTS * 8 * kFrag) + (size_t)w * 2 * kFrag;
    const unsigned ldo = (unsigned)(p.Hv * p.dv);
    T* op = (T*)a.o + (size_t)at.r.start * ldo + (size_t)at.h * p.dv;
    unsigned ooff[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) ooff[e] = (unsigned)(i0 + e) * ldo + at.ccol;
    auto load_p = [&] {
      ev = *reinterpret_cast<const v4f*>(dp->e + i0);
#pragma unroll
      for (int q = 0; q < OUTS; ++q) pa[0][q] = load_frag(pp, q * 8, off);
      if (w >= 2)
#pragma unroll
        for (int q = 0; q < OUTS; ++q) pa[1][q] = load_frag(pp, q * 8 + 1, off);
    };
    if (nc > 0) load_p();
    for (int c = 0; c < nc; ++c) {
      if (c + 1 < nc) {
        pp += (size_t)p.Hv * (OUTS * 8 * kFrag);
        dp += p.Hv;
      }
      __syncthreads();
      __syncthreads();
      v4f o = *reinterpret_cast<const v4f*>(&pq[0][lr][i0]);
#pragma unroll
      for (int i = 1; i < O::WAVES; ++i) o += *reinterpret_cast<const v4f*>(&pq[i][lr][i0]);
      o *= ev * a.scale;
      __syncthreads();
      v8bf ub[OUTS];
      get8<OUTS>(ut, ub, lr, lg * 8);
      o = mfma_parts<OUTS>(pa[0], ub, o);
      if (w >= 2) {
        get8<OUTS>(ut, ub, lr, 32 + lg * 8);
        o = mfma_parts<OUTS>(pa[1], ub, o);
      }
      load_p();
      const int n = (int)(at.r.len - (long)c * kChunk);
      if (at.colon) {
        if (n >= kChunk) {
#pragma unroll
          for (int e = 0; e < 4; ++e) op[ooff[e]] = from_f32<T>(o[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i0 + e < n) op[ooff[e]] = from_f32<T>(o[e]);
        }
      }
      op += (size_t)kChunk * ldo;
    }
  }
}

// The same backwards, for the gradient Z of the state behind a chunk (dS' in the
// formulas):
//   dU = (scale P)^T dO + d . (K Z),  dV = X^T (beta . dU),
//   Z <- e_last Z + Q^T (scale e . dO) - K^T (e . dV).
// Waves 0 - 3 walk this chain; waves 4 - 7 prepare the products with dO a chunk
// ahead and store dV (the gradient of v, and fp32 [dv][64] for stage 3).  Z before
// its update is kept for stage 3.
template <typename T, int PARTS, int OUTS, int DKP>
__global__ __launch_bounds__(512) void delta_scan_bwd_kernel(const s4dplr_delta_plan p,
                                                             const DeltaArgs a) {
  using O = Own<DKP>;
  constexpr int KS = O::KS, KW = O::KW, RT = O::RT;
  __shared__ __attribute__((aligned(16))) float pk[O::WAVES][DS][kLdF];   // K Z, by owner
  __shared__ __attribute__((aligned(16))) float d1[2][DS][kLdF];          // (scale P)^T dO
  __shared__ __attribute__((aligned(16))) float vs[DS][kLdF];             // dV
  __shared__ __attribute__((aligned(16))) __bf16 ot[PARTS][DS][kLdT];     // dO
  __shared__ __attribute__((aligned(16))) __bf16 et[2][3][DS][kLdT];      // scale e . dO
  __shared__ __attribute__((aligned(16))) __bf16 ut[3][DS][kLdT];         // beta . dU
  __shared__ __attribute__((aligned(16))) __bf16 vt[3][DS][kLdT];         // -e . dV
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Place at;
  if (!place_of(p, a, lane, &at)) return;
  const int lr = at.lr, lg = at.lg, w = wave & 3, i0 = 16 * w + 4 * lg, nc = at.nc;
  constexpr size_t kbytes = (size_t)PARTS * 4 * KS * kFrag;
  const long slot1 = at.slot0 + nc - 1;   // the last chunk
  const size_t k0 = ((size_t)slot1 * p.Hk + at.hk) * kbytes;
  const size_t v0 = (size_t)slot1 * p.Hv + at.h;
  const size_t kstep = (size_t)p.Hk * kbytes;
  const unsigned off = lane * 16;
  const DeltaVec* dp = reinterpret_cast<const DeltaVec*>(a.ws + p.off_vec) + v0;
  const v4f zero = {0.f, 0.f, 0.f, 0.f};

  if (wave < 4) {
    __builtin_amdgcn_s_setprio(1);
    const int kw = O::kw(w) * KW, rt0 = O::rt(w);
    v4f Z[KW][2];
    load_state<KW>(Z, a.dstate_out, kw, p, at);
    if (nc > 0) {
      v8bf ka[KW][RT][PARTS], xa[2][3], ta[KW][2][2][PARTS], qa[KW][2][2][PARTS];
      v4f ev, dv, bv;
      float el;
      const unsigned char* kp = a.ws + p.off_k + k0 + (size_t)(rt0 * KS + kw) * kFrag;
      const unsigned char* tp = a.ws + p.off_kt + k0 + (size_t)kw * 4 * kFrag;
      const unsigned char* qp = a.ws + p.off_qt + k0 + (size_t)kw * 4 * kFrag;
      const unsigned char* xp = a.ws + p.off_x + v0 * (3 * 8 * kFrag) + (size_t)w * 2 * kFrag;
      float* zp = reinterpret_cast<float*>(a.ws + p.off_ds) + v0 * p.dk * p.dv +
                  (size_t)at.ccol * p.dk;
      auto load_k = [&] {
#pragma unroll
        for (int q = 0; q < PARTS; ++q)
#pragma unroll
          for (int t = 0; t < RT; ++t)
#pragma unroll
            for (int i = 0; i < KW; ++i) ka[i][t][q] = load_frag(kp, (q * 4 + t) * KS + i, off);
      };
      auto load_x = [&] {   // X^T: upper
#pragma unroll
        for (int i = 0; i < 3; ++i) xa[1][i] = load_frag(xp, i * 8 + 1, off);
        if (w < 2)
#pragma unroll
          for (int i = 0; i < 3; ++i) xa[0][i] = load_frag(xp, i * 8, off);
      };
      auto load_t = [&](const unsigned char* from, v8bf (&to)[KW][2][2][PARTS]) {
#pragma unroll
        for (int q = 0; q < PARTS; ++q)
#pragma unroll
          for (int i = 0; i < KW; ++i)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int ks = 0; ks < 2; ++ks)
                to[i][t][ks][q] = load_frag(from, (q * (DKP / 16) + 2 * i + t) * 2 + ks, off);
      };
      auto load_d = [&] {
        ev = *reinterpret_cast<const v4f*>(dp->e + i0);
        dv = *reinterpret_cast<const v4f*>(dp->d + i0);
        bv = *reinterpret_cast<const v4f*>(dp->beta + i0);
        el = dp->e[kChunk - 1];
      };
      load_k();
      load_d();
      load_x();
      load_t(qp, qa);
      load_t(tp, ta);
      __syncthreads();   // the others' first products
      __syncthreads();
      for (int c = nc - 1; c >= 0; --c) {
        if (c > 0) {   // else the same operands once more
          kp -= kstep;
          qp -= kstep;
          tp -= kstep;
          xp -= (size_t)p.Hv * (3 * 8 * kFrag);
          dp -= p.Hv;
        }
        const int b = c & 1;
        {
          v4f x[RT];
#pragma unroll
          for (int t = 0; t < RT; ++t) x[t] = zero;
#pragma unroll
          for (int i = 0; i < KW; ++i) {
            v8bf sb[3];
            state_operand(Z[i], sb);
#pragma unroll
            for (int t = 0; t < RT; ++t) x[t] = mfma_parts<3>(ka[i][t], sb, x[t]);
          }
          if (at.colon && O::first(w)) keep_state<KW>(Z, zp, kw, p.dk, lg);
          zp -= (size_t)p.Hv * p.dk * p.dv;
#pragma unroll
          for (int t = 0; t < RT; ++t)
            *reinterpret_cast<v4f*>(&pk[O::kw(w)][lr][16 * (rt0 + t) + 4 * lg]) = x[t];
        }
        load_k();
        __syncthreads();
        {
          v4f kz = *reinterpret_cast<const v4f*>(&pk[0][lr][i0]);
#pragma unroll
          for (int i = 1; i < O::WAVES; ++i) kz += *reinterpret_cast<const v4f*>(&pk[i][lr][i0]);
          const v4f g = *reinterpret_cast<const v4f*>(&d1[b][lr][i0]);
          put4<3>(ut, bv * (g + dv * kz), lr, i0);
        }
        // off the chain: Q^T (scale e . dO)
#pragma unroll
        for (int i = 0; i < KW; ++i)
#pragma unroll
          for (int t = 0; t < 2; ++t) Z[i][t] *= el;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          v8bf eb[3];
          get8<3>(et[b], eb, lr, ks * 32 + lg * 8);
#pragma unroll
          for (int i = 0; i < KW; ++i)
#pragma unroll
            for (int t = 0; t < 2; ++t) Z[i][t] = mfma_parts<3>(qa[i][t][ks], eb, Z[i][t]);
        }
        __syncthreads();
        v4f dV = zero, dV1 = zero;
        {
          v8bf ub[3], uc[3];
          get8<3>(ut, ub, lr, 32 + lg * 8);
          if (w < 2) {
            get8<3>(ut, uc, lr, lg * 8);
            dV1 = mfma_parts<3>(xa[0], uc, dV1);
          }
          dV = mfma_parts<3>(xa[1], ub, dV);
          dV += dV1;
        }
        put4<3>(vt, -(ev * dV), lr, i0);
        *reinterpret_cast<v4f*>(&vs[lr][i0]) = dV;
        load_t(qp, qa);
        load_x();
        load_d();
        __syncthreads();
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          v8bf vb[3];
          get8<3>(vt, vb, lr, ks * 32 + lg * 8);
#pragma unroll
          for (int i = 0; i < KW; ++i)
#pragma unroll
            for (int t = 0; t < 2; ++t) Z[i][t] = mfma_parts<3>(ta[i][t][ks], vb, Z[i][t]);
        }
        load_t(tp, ta);
      }
    }
    if (O::first(w)) store_state<KW>(Z, a.dstate, kw, p, at);
  } else if (nc > 0) {
    v8bf pa[2][OUTS];
    v4f ev;
    T go[4];
    const unsigned char* pp = a.ws + p.off_p + v0 * (OUTS * 8 * kFrag) + (size_t)w * 2 * kFrag;
    const unsigned ldo = (unsigned)(p.Hv * p.dv);
    const size_t row1 = (size_t)at.r.start + (size_t)(nc - 1) * kChunk;
    const T* gp = (const T*)a.dout + row1 * ldo + (size_t)at.h * p.dv;
    T* op = (T*)a.dv + row1 * ldo + (size_t)at.h * p.dv;
    float* fp = reinterpret_cast<float*>(a.ws + p.off_dv) + v0 * kChunk * p.dv +
                (size_t)at.ccol * kChunk + i0;
    unsigned ooff[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) ooff[e] = (unsigned)(i0 + e) * ldo + at.ccol;
    auto rows = [&](int c) { return (int)(at.r.len - (long)c * kChunk); };
    auto load = [&](int c) {   // chunk c's, by the moving pointers
      ev = *reinterpret_cast<const v4f*>(dp->e + i0);
      const int n = rows(c);
      if (n >= kChunk) {
#pragma unroll
        for (int e = 0; e < 4; ++e) go[e] = ((const GLOBAL T*)gp)[ooff[e]];
      } else {   // rows behind the end: Q and P are zero there
#pragma unroll
        for (int e = 0; e < 4; ++e)
          go[e] = ((const GLOBAL T*)gp)[(unsigned)(i0 + e < n ? i0 + e : n - 1) * ldo + at.ccol];
      }
#pragma unroll
      for (int q = 0; q < OUTS; ++q) pa[1][q] = load_frag(pp, q * 8 + 1, off);
      if (w < 2)
#pragma unroll
        for (int q = 0; q < OUTS; ++q) pa[0][q] = load_frag(pp, q * 8, off);
    };
    auto put = [&](int c) {
      v4f g;
#pragma unroll
      for (int e = 0; e < 4; ++e) g[e] = to_f32(go[e]);
      put4<PARTS>(ot, g, lr, i0);
      put4<3>(et[c & 1], g * (ev * a.scale), lr, i0);
    };
    auto product = [&](int c) {
      v4f g = zero;
      v8bf ob[PARTS];
      get8<PARTS>(ot, ob, lr, 32 + lg * 8);
      g = mfma_parts<3>(pa[1], ob, g);
      if (w < 2) {
        get8<PARTS>(ot, ob, lr, lg * 8);
        g = mfma_parts<3>(pa[0], ob, g);
      }
      *reinterpret_cast<v4f*>(&d1[c & 1][lr][i0]) = g;
    };
    auto back = [&](int c) {   // to chunk c - 1
      if (c > 0) {
        pp -= (size_t)p.Hv * (OUTS * 8 * kFrag);
        gp -= (size_t)kChunk * ldo;
        dp -= p.Hv;
      }
      load(c > 0 ? c - 1 : 0);
    };
    load(nc - 1);
    put(nc - 1);
    __syncthreads();
    product(nc - 1);
    back(nc - 1);
    __syncthreads();
    for (int c = nc - 1; c >= 0; --c) {
      __syncthreads();
      put(c + 1);        // chunk c - 1's slot: the parity of c + 1
      __syncthreads();
      product(c + 1);
      back(c > 0 ? c - 1 : 0);
      __syncthreads();
      const v4f dV = *reinterpret_cast<const v4f*>(&vs[lr][i0]);
      if (at.colon) {
        *reinterpret_cast<v4f*>(fp) = dV;
        if (a.dv) {
          const int n = rows(c);
          if (n >= kChunk) {
#pragma unroll
            for (int e = 0; e < 4; ++e) op[ooff[e]] = from_f32<T>(dV[e]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (i0 + e < n) op[ooff[e]] = from_f32<T>(dV[e]);
          }
        }
      }
      fp -= (size_t)p.Hv * kChunk * p.dv;
      op -= (size_t)kChunk * ldo;
    }
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
    delta_scan_bwd_kernel<T, PARTS, OUTS, dkp><<<grid, 512, 0, s>>>(*p, a);            \
  else if (a.saved)                                                                    \
    delta_scan_kernel<T, PARTS, OUTS, dkp, true><<<grid, 512, 0, s>>>(*p, a);          \
  else                                                                                 \
    delta_scan_kernel<T, PARTS, OUTS, dkp, false><<<grid, 512, 0, s>>>(*p, a)
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
