// Gated delta rule, chunked form, stage 2: the chunks of a sequence one after
// another.  A block carries DS = 16 or 32 columns of one head's dk x dv state S through
// them:
//   R = V - e . (K S),  N = X R,  U = beta . N,
//   O = scale e . (Q S) + (scale P) U,  S <- e_last S + K^T (d . U).
//
// A step is a chain of small products with an exchange between waves after each,
// so its time is latency and instruction issue, not bandwidth (256 chunks after one
// another, 16 heads of 128 x 128 in bf16: 466 us forward, 1.8 us a chunk; 4 sequences of 64
// chunks: 317 us forward with N and S saved, 295 us backward).  Of the 8 waves, 0 - 3
// walk the chain: wave w owns a quarter of S's rows in fp32 accumulators.  K^T is
// stored with its rows permuted so that the two accumulator tiles of 32 rows hold 8
// neighbouring rows a lane: a matrix operand's layout, so S enters K S straight from
// registers as three bf16 parts; the waves' partial sums meet in LDS.  R and d . U pass
// through LDS as bf16 parts.  Waves 4, 5 compute O beside the chain.  Waves 6, 7 only
// store (a wave that stores waits for its stores before loads that it issued behind
// them) and touch the operands three chunks ahead, a line a lane, since a step is
// shorter than a load from HBM takes: the chain's own loads then hit the XCD's L2,
// which the slices of a head share (each touches its part).  Row tiles of X and K^T
// belong to one wave each: those operands go from memory to registers, a chunk ahead.
#include "delta_device.h"

namespace s4 {

namespace {

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
  __device__ __forceinline__ int col(int u) const { return col0 + 16 * u + lr; }
  int sh, h, hk, nc, slice, slices, col0, lr, lg;
  Rows r;
  long slot0;
};
template <int DS>
__device__ __forceinline__ bool place_of(const s4dplr_delta_plan& p, const DeltaArgs& a, int lane,
                                         Place* o) {
  o->slices = (p.dv + DS - 1) / DS;
  if (!slice_of(p.sequences * p.Hv, o->slices, &o->sh, &o->slice)) return false;
  const int s = o->sh / p.Hv;
  o->h = o->sh % p.Hv;
  o->hk = o->h / (p.Hv / p.Hk);
  o->r = rows_of(p, a.offsets, s);
  o->nc = o->r.chunks();
  o->slot0 = o->r.first(s, a.least);
  o->lr = lane & 15;
  o->lg = lane >> 4;
  o->col0 = o->slice * DS;
  return true;
}

// The wave's rows of a state [dk][dv] in fp32: tile t of k step k, accumulator entry e,
// is row 32 k + 8 lg + 4 t + e.
template <int KW>
__device__ __forceinline__ void load_state(v4f (&S)[KW][2], const float* state, int k0, int col,
                                           const s4dplr_delta_plan& p, const Place& at) {
#pragma unroll
  for (int i = 0; i < KW; ++i)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = 32 * (k0 + i) + 8 * at.lg + 4 * t + e;
        S[i][t][e] = state && col < p.dv && d < p.dk
                         ? state[((size_t)at.sh * p.dk + d) * p.dv + col] : 0.f;
      }
}
template <int KW>
__device__ __forceinline__ void store_state(const v4f (&S)[KW][2], float* state, int k0, int col,
                                            const s4dplr_delta_plan& p, const Place& at) {
  if (!state || col >= p.dv) return;
#pragma unroll
  for (int i = 0; i < KW; ++i)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = 32 * (k0 + i) + 8 * at.lg + 4 * t + e;
        if (d < p.dk) state[((size_t)at.sh * p.dk + d) * p.dv + col] = S[i][t][e];
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

template <int N, int DS>
__device__ __forceinline__ void put4(__bf16 (*to)[DS][kLdT], v4f x, int lr, int i0) {
  v4bf t[N];
  split4<N>(x, t);
#pragma unroll
  for (int q = 0; q < N; ++q) *reinterpret_cast<v4bf*>(&to[q][lr][i0]) = t[q];
}
template <int N, int DS>
__device__ __forceinline__ void get8(const __bf16 (*from)[DS][kLdT], v8bf (&x)[N], int lr, int k) {
#pragma unroll
  for (int q = 0; q < N; ++q) x[q] = *reinterpret_cast<const v8bf*>(&from[q][lr][k]);
}

// The storing waves: j = 0, 1.  A matrix [DS][LD] in LDS to [dv][n] in memory (`to`:
// the slice's first column), rows of n floats.
template <int LD, int DS>
__device__ __forceinline__ void store_columns(float* to, const float (&m)[DS][LD], int n, int cols,
                                              int j, int lane) {
  constexpr int G = (LD - 4) / 4;   // groups of 4 a column
#pragma unroll
  for (int i = 0; i < DS * G / 128; ++i) {
    const int at = (i * 2 + j) * 64 + lane, c = at / G, d = at % G * 4;
    const v4f x = *reinterpret_cast<const v4f*>(&m[c][d]);
    if (c >= cols) continue;
    float* t = to + (unsigned)(c * n + d);
    if (d + 4 <= n) {
      __builtin_memcpy(t, &x, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (d + e < n) t[e] = x[e];
    }
  }
}
// The state's columns from its three parts in LDS (their sum is exact) to [dv][dk].
template <int DKP, int DS>
__device__ __forceinline__ void store_parts(float* to, const __bf16 (*m)[DS][DKP + 8], int dk,
                                            int cols, int j, int lane) {
#pragma unroll
  for (int i = 0; i < DS * DKP / 8 / 128; ++i) {
    const int at = (i * 2 + j) * 64 + lane, c = at / (DKP / 8), d = at % (DKP / 8) * 8;
    const v8bf x = *reinterpret_cast<const v8bf*>(&m[0][c][d]);
    const v8bf y = *reinterpret_cast<const v8bf*>(&m[1][c][d]);
    const v8bf z = *reinterpret_cast<const v8bf*>(&m[2][c][d]);
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = (float)x[e] + ((float)y[e] + (float)z[e]);
    if (c < cols) store8(to + (unsigned)(c * dk + d), dk - d, t);
  }
}
// A chunk's rows from LDS [column][row] to memory: 8 columns of one row a lane.
template <typename T, int DS>
__device__ __forceinline__ void store_rows(T* to, unsigned ld, const float (&m)[DS][kLdF], int cols,
                                           int n, int j, int lane) {
  constexpr int G = DS / 8;   // lanes a row
#pragma unroll
  for (int i = 0; i < DS / 16; ++i) {
    const int at = (i * 2 + j) * 64 + lane, row = at / G, c = at % G * 8;
    T t[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) t[q] = from_f32<T>(m[c + q][row]);
    if (row >= n) continue;
    T* o = to + (unsigned)(row * ld + c);
    if (c + 8 <= cols) {
      __builtin_memcpy(o, t, sizeof(t));
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c + q < cols) o[q] = t[q];
    }
  }
}

// Lines of a chunk's operands to bring into the L2: K, then Q (forward) or Q^T
// (backward), K^T, X, P, shared among the slices of a head; and the slice's own rows
// of V or dO with the decays.  Chunks are counted from the sequence's first.
template <int PARTS, int DKP, bool BWD>
struct Ahead {
  static constexpr int kTouch = 5;            // lines a lane and chunk, at most
  static constexpr int kSets = 4;             // chunks in flight
  static constexpr int KL = PARTS * DKP;      // lines of a 64 x DKP operand (128 bytes each)
  static constexpr int XL = 3 * 8 * kFrag / 128;   // lines of X, and of P
  static constexpr int kLines = 3 * KL + 2 * XL;
  const unsigned char *k, *q, *t, *x, *p, *v, *d;
  long ldv;                                   // bytes from row to row of V or dO
  size_t kstep, xstep, dstep;
  int id, first, step;                        // this lane's lines: first + i step
  static constexpr int kSize = PARTS == 3 ? 4 : 2;   // bytes of an element

  __device__ __forceinline__ void set(const s4dplr_delta_plan& pl, const DeltaArgs& a,
                                      const Place& at, int lane) {
    constexpr size_t kbytes = (size_t)KL * 128;
    const size_t f = ((size_t)at.slot0 * pl.Hk + at.hk) * kbytes;
    const size_t g = (size_t)at.slot0 * pl.Hv + at.h;
    k = a.ws + pl.off_k + f;
    q = a.ws + (BWD ? pl.off_qt : pl.off_q) + f;
    t = a.ws + pl.off_kt + f;
    x = a.ws + pl.off_x + g * (XL * 128);
    p = a.ws + pl.off_p + g * (XL * 128);
    v = (const unsigned char*)(BWD ? a.dout : a.v);
    ldv = (BWD ? (long)pl.Hv * pl.dv : a.ldv) * kSize;
    v += at.r.start * ldv + ((size_t)at.h * pl.dv + at.col0) * kSize;
    d = a.ws + pl.off_vec + g * sizeof(DeltaVec);
    dstep = (size_t)pl.Hv * sizeof(DeltaVec);
    id = lane;
    kstep = (size_t)pl.Hk * kbytes;
    xstep = (size_t)pl.Hv * (XL * 128);
    first = at.slice * 128 + lane;
    step = at.slices * 128;
  }
  // A whole chunk c.
  __device__ __forceinline__ void touch(long c, unsigned (&h)[kTouch]) const {
#pragma unroll
    for (int i = 0; i < kTouch - 1; ++i) {
      if (i * step >= kLines) continue;   // uniform
      int l = first + i * step;
      if (l >= kLines) l = 0;
      const unsigned char* from;
      if (l < KL) {
        from = k + c * (long)kstep + l * 128;
      } else if ((l -= KL) < KL) {
        from = q + c * (long)kstep + l * 128;
      } else if ((l -= KL) < KL) {
        from = t + c * (long)kstep + l * 128;
      } else if ((l -= KL) < XL) {
        from = x + c * (long)xstep + l * 128;
      } else {
        from = p + c * (long)xstep + (l - XL) * 128;
      }
      h[i] = *(const GLOBAL unsigned char*)from;
    }
    const long line = id - 64 < (int)sizeof(DeltaVec) / 128 ? id - 64 : 0;
    const unsigned char* from =
        id < 64 ? v + (c * 64 + id) * ldv : d + c * (long)dstep + line * 128;
    h[kTouch - 1] = *(const GLOBAL unsigned char*)from;
  }
  // What was touched some chunks ago has to have arrived: its registers are free again.
  __device__ static __forceinline__ void settle(const unsigned (&h)[kTouch]) {
#pragma unroll
    for (int i = 0; i < kTouch; ++i) asm volatile("" ::"v"(h[i]));
  }
};

}  // namespace

template <typename T, int PARTS, int DKP, bool SAVE, int DS>
__global__ __launch_bounds__(512) void delta_scan_kernel(const s4dplr_delta_plan p,
                                                         const DeltaArgs a) {
  using O = Own<DKP>;
  constexpr int KS = O::KS, KW = O::KW, RT = O::RT, NT = DS / 16;   // NT: column tiles
  __shared__ __attribute__((aligned(16))) float pk[O::WAVES][DS][kLdF];   // K S, by owner
  __shared__ __attribute__((aligned(16))) float os[DS][kLdF];             // O
  __shared__ __attribute__((aligned(16))) float ns[SAVE ? DS : 1][kLdF];  // N
  __shared__ __attribute__((aligned(16))) __bf16 st[3][DS][DKP + 8];      // S
  __shared__ __attribute__((aligned(16))) __bf16 rt[3][DS][kLdT];         // R
  __shared__ __attribute__((aligned(16))) __bf16 ut[3][DS][kLdT];      // U
  __shared__ __attribute__((aligned(16))) __bf16 du[3][DS][kLdT];         // d . U
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Place at;
  if (!place_of<DS>(p, a, lane, &at) || at.r.len <= a.step_tokens) return;
  const int lr = at.lr, lg = at.lg, nc = at.nc;
  constexpr size_t kbytes = (size_t)PARTS * 4 * KS * kFrag;
  const size_t k0 = ((size_t)at.slot0 * p.Hk + at.hk) * kbytes;
  const size_t v0 = (size_t)at.slot0 * p.Hv + at.h;
  const size_t kstep = (size_t)p.Hk * kbytes;
  const unsigned off = lane * 16;
  const DeltaVec* dp = reinterpret_cast<const DeltaVec*>(a.ws + p.off_vec) + v0;
  const v4f zero = {0.f, 0.f, 0.f, 0.f};

  if (wave < 4) {
    __builtin_amdgcn_s_setprio(1);
    const int w = wave, i0 = 16 * w + 4 * lg, kw = O::kw(w) * KW, rt0 = O::rt(w);
    v4f S[NT][KW][2];
#pragma unroll
    for (int u = 0; u < NT; ++u) load_state<KW>(S[u], a.state, kw, at.col(u), p, at);

    // Operands of one chunk, each set loaded right after its last use.
    v8bf ka[KW][RT][PARTS], xa[2][3], ta[KW][2][2][PARTS];
    v4f ev, dv, bv;
    float el;
    T vv[NT][4];
    const unsigned char* kp = a.ws + p.off_k + k0 + (size_t)(rt0 * KS + kw) * kFrag;
    const unsigned char* tp = a.ws + p.off_kt + k0 + (size_t)kw * 4 * kFrag;
    const unsigned char* xp = a.ws + p.off_x + v0 * (3 * 8 * kFrag) + (size_t)w * 2 * kFrag;
    const T* vp = (const T*)a.v + at.r.start * a.ldv + (size_t)at.h * p.dv;
    const unsigned ldv = (unsigned)a.ldv;
    // columns behind dv read column 0: nothing of theirs is stored
    unsigned voff[4], vcol[NT];
#pragma unroll
    for (int e = 0; e < 4; ++e) voff[e] = (unsigned)(i0 + e) * ldv;
#pragma unroll
    for (int u = 0; u < NT; ++u) vcol[u] = at.col(u) < p.dv ? at.col(u) : 0;
    auto load_k = [&] {
#pragma unroll
      for (int q = 0; q < PARTS; ++q)
#pragma unroll
        for (int t = 0; t < RT; ++t)
#pragma unroll
          for (int i = 0; i < KW; ++i) ka[i][t][q] = load_frag(kp, (q * 4 + t) * KS + i, off);
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
    auto load_v = [&](int n) {
      if (n >= kChunk) {
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) vv[u][e] = vp[voff[e] + vcol[u]];
      } else {
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            vv[u][e] = vp[(unsigned)(i0 + e < n ? i0 + e : n - 1) * ldv + vcol[u]];
      }
    };
    auto load_d = [&] {
      ev = *reinterpret_cast<const v4f*>(dp->e + i0);
      dv = *reinterpret_cast<const v4f*>(dp->d + i0);
      bv = *reinterpret_cast<const v4f*>(dp->beta + i0);
      el = dp->e[kChunk - 1];
    };
    int n = (int)at.r.len;   // rows left from the loaded chunk on
    if (nc > 0) {
      load_k();
      load_v(n);
      load_d();
      load_x();
      load_t();
    }
    for (int c = 0; c < nc; ++c) {
      if (c + 1 < nc) {   // else the same operands once more
        n -= kChunk;
        kp += kstep;
        tp += kstep;
        xp += (size_t)p.Hv * (3 * 8 * kFrag);
        dp += p.Hv;
        vp += (size_t)kChunk * ldv;
      }
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        v4f x[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) x[t] = zero;
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          v8bf sb[3];
          state_operand(S[u][i], sb);
#pragma unroll
          for (int t = 0; t < RT; ++t) x[t] = mfma_parts<3>(ka[i][t], sb, x[t]);
          if (O::first(w))
#pragma unroll
            for (int q = 0; q < 3; ++q)
              *reinterpret_cast<v8bf*>(&st[q][16 * u + lr][32 * (kw + i) + 8 * lg]) = sb[q];
        }
#pragma unroll
        for (int t = 0; t < RT; ++t)
          *reinterpret_cast<v4f*>(&pk[O::kw(w)][16 * u + lr][16 * (rt0 + t) + 4 * lg]) = x[t];
      }
      __syncthreads();
      load_k();
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        v4f sum = *reinterpret_cast<const v4f*>(&pk[0][16 * u + lr][i0]);
#pragma unroll
        for (int i = 1; i < O::WAVES; ++i)
          sum += *reinterpret_cast<const v4f*>(&pk[i][16 * u + lr][i0]);
        v4f R;
#pragma unroll
        for (int e = 0; e < 4; ++e) R[e] = to_f32(vv[u][e]);
        put4<3>(rt, R - ev * sum, 16 * u + lr, i0);
      }
      load_v(n);
      __syncthreads();
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        v4f N = zero, n1 = zero;
        v8bf rb[3], rc[3];
        get8<3>(rt, rb, 16 * u + lr, lg * 8);
        if (w >= 2) {
          get8<3>(rt, rc, 16 * u + lr, 32 + lg * 8);
          n1 = mfma_parts<3>(xa[1], rc, n1);
        }
        N = mfma_parts<3>(xa[0], rb, N);
        N += n1;
        const v4f U = bv * N;
        put4<3>(du, dv * U, 16 * u + lr, i0);
        put4<3>(ut, U, 16 * u + lr, i0);
        if constexpr (SAVE) *reinterpret_cast<v4f*>(&ns[16 * u + lr][i0]) = N;
      }
      load_x();
      __syncthreads();
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        v8bf ub[2][3];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) get8<3>(du, ub[ks], 16 * u + lr, ks * 32 + lg * 8);
#pragma unroll
        for (int i = 0; i < KW; ++i)
#pragma unroll
          for (int t = 0; t < 2; ++t) S[u][i][t] *= el;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int i = 0; i < KW; ++i)
#pragma unroll
            for (int t = 0; t < 2; ++t)
              S[u][i][t] = mfma_parts<3>(ta[i][t][ks], ub[ks], S[u][i][t]);
      }
      load_d();
      load_t();
    }
    __syncthreads();
    if (O::first(w))
#pragma unroll
      for (int u = 0; u < NT; ++u) store_state<KW>(S[u], a.state_out, kw, at.col(u), p, at);
  } else if (wave < 6) {
    // row tiles j and 3 - j of O: one of them reaches over both k steps of P
    const int j = wave - 4;
    v8bf p0[3], p1[2][3], qa[2][KS][PARTS];
    v4f ev[2];
    const unsigned char* qp = a.ws + p.off_q + k0;
    const unsigned char* pp = a.ws + p.off_p + v0 * (3 * 8 * kFrag);
    auto load_q = [&] {
#pragma unroll
      for (int q = 0; q < PARTS; ++q)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          qa[0][ks][q] = load_frag(qp + (size_t)j * KS * kFrag, q * 4 * KS + ks, off);
          qa[1][ks][q] = load_frag(qp + (size_t)(3 - j) * KS * kFrag, q * 4 * KS + ks, off);
        }
      ev[0] = *reinterpret_cast<const v4f*>(dp->e + 16 * j + 4 * lg);
      ev[1] = *reinterpret_cast<const v4f*>(dp->e + 16 * (3 - j) + 4 * lg);
    };
    auto load_p = [&] {
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        p0[q] = load_frag(pp + (size_t)j * 2 * kFrag, q * 8, off);
        p1[0][q] = load_frag(pp + (size_t)(3 - j) * 2 * kFrag, q * 8, off);
        p1[1][q] = load_frag(pp + (size_t)(3 - j) * 2 * kFrag, q * 8 + 1, off);
      }
    };
    if (nc > 0) {
      load_q();
      load_p();
    }
    for (int c = 0; c < nc; ++c) {
      if (c + 1 < nc) {
        qp += kstep;
        pp += (size_t)p.Hv * (3 * 8 * kFrag);
        dp += p.Hv;
      }
      __syncthreads();
      v4f o[NT][2];
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        o[u][0] = o[u][1] = zero;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          v8bf sb[3];
#pragma unroll
          for (int q = 0; q < 3; ++q)
            sb[q] = *reinterpret_cast<const v8bf*>(&st[q][16 * u + lr][32 * ks + 8 * lg]);
          o[u][0] = mfma_parts<3>(qa[0][ks], sb, o[u][0]);
          o[u][1] = mfma_parts<3>(qa[1][ks], sb, o[u][1]);
        }
        o[u][0] *= ev[0] * a.scale;
        o[u][1] *= ev[1] * a.scale;
      }
      load_q();
      __syncthreads();
      __syncthreads();
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        v8bf ub[2][3];
        get8<3>(ut, ub[0], 16 * u + lr, lg * 8);
        get8<3>(ut, ub[1], 16 * u + lr, 32 + lg * 8);
        o[u][0] = mfma_parts<3>(p0, ub[0], o[u][0]);
        o[u][1] = mfma_parts<3>(p1[0], ub[0], o[u][1]);
        o[u][1] = mfma_parts<3>(p1[1], ub[1], o[u][1]);
        *reinterpret_cast<v4f*>(&os[16 * u + lr][16 * j + 4 * lg]) = o[u][0];
        *reinterpret_cast<v4f*>(&os[16 * u + lr][16 * (3 - j) + 4 * lg]) = o[u][1];
      }
      load_p();
    }
    __syncthreads();
  } else {
    const int j = wave - 6, cols = p.dv - at.col0;
    const unsigned ldo = (unsigned)(p.Hv * p.dv);
    T* op = (T*)a.o + (size_t)at.r.start * ldo + (size_t)at.h * p.dv + at.col0;
    float *np = nullptr, *sp = nullptr;
    if constexpr (SAVE) {
      np = reinterpret_cast<float*>(a.saved + p.off_n) + (v0 * p.dv + at.col0) * kChunk;
      sp = reinterpret_cast<float*>(a.saved + p.off_s) + (v0 * p.dv + at.col0) * p.dk;
    }
    using A = Ahead<PARTS, DKP, false>;
    A ahead;
    ahead.set(p, a, at, j * 64 + lane);
    const int whole = (int)(at.r.len / kChunk);
    // chunks behind the last whole one are not touched: their rows need not exist
    auto touch = [&](int c, unsigned (&h)[A::kTouch]) {
      if (c < whole) ahead.touch(c, h);
    };
    unsigned held[A::kSets][A::kTouch] = {};
    touch(1, held[1]);
    touch(2, held[2]);
    for (int c4 = 0; c4 < nc; c4 += A::kSets)
#pragma unroll
      for (int u = 0; u < A::kSets; ++u) {
        const int c = c4 + u;
        if (c < nc) {
          A::settle(held[(u + 3) % A::kSets]);
          touch(c + 3, held[(u + 3) % A::kSets]);
          __syncthreads();
          if constexpr (SAVE) {
            store_parts<DKP>(sp, st, p.dk, cols, j, lane);
            sp += (size_t)p.Hv * p.dk * p.dv;
          }
          if (c > 0) {
            store_rows(op, ldo, os, cols, kChunk, j, lane);
            op += (size_t)kChunk * ldo;
          }
          __syncthreads();
          __syncthreads();
          if constexpr (SAVE) {
            store_columns(np, ns, kChunk, cols, j, lane);
            np += (size_t)p.Hv * kChunk * p.dv;
          }
        }
      }
    __syncthreads();
    if (nc > 0) store_rows(op, ldo, os, cols, (int)(at.r.len - (long)(nc - 1) * kChunk), j, lane);
  }
}

// The same backwards, for the gradient Z of the state behind a chunk (dS' in the
// formulas):
//   dU = (scale P)^T dO + d . (K Z),  dV = X^T (beta . dU),
//   Z <- e_last Z + Q^T (scale e . dO) - K^T (e . dV).
// Waves 0 - 3 walk this chain, 4 and 5 prepare the products with dO a chunk ahead, 6
// and 7 store dV (the gradient of v, and fp32 [dv][64] for stage 3) and Z before its
// update ([dv][dk], for stage 3).
template <typename T, int PARTS, int DKP, int DS>
__global__ __launch_bounds__(512) void delta_scan_bwd_kernel(const s4dplr_delta_plan p,
                                                             const DeltaArgs a) {
  using O = Own<DKP>;
  constexpr int KS = O::KS, KW = O::KW, RT = O::RT, NT = DS / 16;   // NT: column tiles
  __shared__ __attribute__((aligned(16))) float pk[O::WAVES][DS][kLdF];   // K Z, by owner
  __shared__ __attribute__((aligned(16))) float d1[2][DS][kLdF];          // (scale P)^T dO
  __shared__ __attribute__((aligned(16))) float vs[DS][kLdF];             // dV
  __shared__ __attribute__((aligned(16))) float ss[DS][DKP + 4];          // Z
  __shared__ __attribute__((aligned(16))) __bf16 ot[PARTS][DS][kLdT];     // dO
  __shared__ __attribute__((aligned(16))) float eq[2][DS][DKP + 4];       // Q^T (scale e . dO)
  __shared__ __attribute__((aligned(16))) __bf16 et[3][DS][kLdT];         // scale e . dO
  __shared__ __attribute__((aligned(16))) __bf16 ut[3][DS][kLdT];         // beta . dU
  __shared__ __attribute__((aligned(16))) __bf16 vt[3][DS][kLdT];         // -e . dV
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Place at;
  if (!place_of<DS>(p, a, lane, &at)) return;
  const int lr = at.lr, lg = at.lg, nc = at.nc;
  constexpr size_t kbytes = (size_t)PARTS * 4 * KS * kFrag;
  const long slot1 = at.slot0 + nc - 1;   // the last chunk
  const size_t k0 = ((size_t)slot1 * p.Hk + at.hk) * kbytes;
  const size_t v0 = (size_t)slot1 * p.Hv + at.h;
  const size_t kstep = (size_t)p.Hk * kbytes;
  const unsigned off = lane * 16;
  const DeltaVec* dp = reinterpret_cast<const DeltaVec*>(a.ws + p.off_vec) + v0;
  const v4f zero = {0.f, 0.f, 0.f, 0.f};
  const unsigned ldo = (unsigned)(p.Hv * p.dv);
  const size_t row1 = (size_t)at.r.start + (size_t)(nc - 1) * kChunk;
  const int last = (int)(at.r.len - (long)(nc - 1) * kChunk);   // rows of the last chunk

  if (wave < 4) {
    __builtin_amdgcn_s_setprio(1);
    const int w = wave, i0 = 16 * w + 4 * lg, kw = O::kw(w) * KW, rt0 = O::rt(w);
    v4f Z[NT][KW][2];
#pragma unroll
    for (int u = 0; u < NT; ++u) load_state<KW>(Z[u], a.dstate_out, kw, at.col(u), p, at);
    if (nc > 0) {
      v8bf ka[KW][RT][PARTS], xa[2][3], ta[KW][2][2][PARTS];
      v4f ev, dv, bv;
      float el;
      const unsigned char* kp = a.ws + p.off_k + k0 + (size_t)(rt0 * KS + kw) * kFrag;
      const unsigned char* tp = a.ws + p.off_kt + k0 + (size_t)kw * 4 * kFrag;
      const unsigned char* xp = a.ws + p.off_x + v0 * (3 * 8 * kFrag) + (size_t)w * 2 * kFrag;
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
      auto load_d = [&] {
        ev = *reinterpret_cast<const v4f*>(dp->e + i0);
        dv = *reinterpret_cast<const v4f*>(dp->d + i0);
        bv = *reinterpret_cast<const v4f*>(dp->beta + i0);
        el = dp->e[kChunk - 1];
      };
      load_k();
      load_d();
      load_x();
      load_t();
      __syncthreads();   // the others' first products
      __syncthreads();
      for (int c = nc - 1; c >= 0; --c) {
        if (c > 0) {   // else the same operands once more
          kp -= kstep;
          tp -= kstep;
          xp -= (size_t)p.Hv * (3 * 8 * kFrag);
          dp -= p.Hv;
        }
        const int b = c & 1;
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          v4f x[RT];
#pragma unroll
          for (int t = 0; t < RT; ++t) x[t] = zero;
#pragma unroll
          for (int i = 0; i < KW; ++i) {
            v8bf sb[3];
            state_operand(Z[u][i], sb);
#pragma unroll
            for (int t = 0; t < RT; ++t) x[t] = mfma_parts<3>(ka[i][t], sb, x[t]);
          }
          if (O::first(w))
#pragma unroll
            for (int i = 0; i < KW; ++i)
#pragma unroll
              for (int t = 0; t < 2; ++t)
                *reinterpret_cast<v4f*>(&ss[16 * u + lr][32 * (kw + i) + 8 * lg + 4 * t]) = Z[u][i][t];
#pragma unroll
          for (int t = 0; t < RT; ++t)
            *reinterpret_cast<v4f*>(&pk[O::kw(w)][16 * u + lr][16 * (rt0 + t) + 4 * lg]) = x[t];
        }
        load_k();
        __syncthreads();
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          v4f kz = *reinterpret_cast<const v4f*>(&pk[0][16 * u + lr][i0]);
#pragma unroll
          for (int i = 1; i < O::WAVES; ++i)
            kz += *reinterpret_cast<const v4f*>(&pk[i][16 * u + lr][i0]);
          const v4f g = *reinterpret_cast<const v4f*>(&d1[b][16 * u + lr][i0]);
          put4<3>(ut, bv * (g + dv * kz), 16 * u + lr, i0);
        }
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int i = 0; i < KW; ++i)
#pragma unroll
            for (int t = 0; t < 2; ++t)
              Z[u][i][t] = Z[u][i][t] * el +
                           *reinterpret_cast<const v4f*>(
                               &eq[b][16 * u + lr][32 * (kw + i) + 8 * lg + 4 * t]);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          v4f dV = zero, dV1 = zero;
          v8bf ub[3], uc[3];
          get8<3>(ut, ub, 16 * u + lr, 32 + lg * 8);
          if (w < 2) {
            get8<3>(ut, uc, 16 * u + lr, lg * 8);
            dV1 = mfma_parts<3>(xa[0], uc, dV1);
          }
          dV = mfma_parts<3>(xa[1], ub, dV);
          dV += dV1;
          put4<3>(vt, -(ev * dV), 16 * u + lr, i0);
          *reinterpret_cast<v4f*>(&vs[16 * u + lr][i0]) = dV;
        }
        load_x();
        load_d();
        __syncthreads();
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            v8bf vb[3];
            get8<3>(vt, vb, 16 * u + lr, ks * 32 + lg * 8);
#pragma unroll
            for (int i = 0; i < KW; ++i)
#pragma unroll
              for (int t = 0; t < 2; ++t)
                Z[u][i][t] = mfma_parts<3>(ta[i][t][ks], vb, Z[u][i][t]);
          }
        load_t();
      }
    }
    if (O::first(w))
#pragma unroll
      for (int u = 0; u < NT; ++u) store_state<KW>(Z[u], a.dstate, kw, at.col(u), p, at);
  } else if (nc > 0 && wave < 6) {
    // row tiles j and 3 - j: one of them reaches over both k steps of P^T
    const int j = wave - 4, ra = 16 * j + 4 * lg, rb = 16 * (3 - j) + 4 * lg;
    constexpr int QT = DKP / 32;   // tiles of Q^T a wave
    v8bf p0[2][3], p1[3], qa[QT][2][PARTS];
    v4f ev[2];
    T go[NT][2][4];
    const unsigned char* qp = a.ws + p.off_qt + k0 + (size_t)j * QT * 2 * kFrag;
    const unsigned char* pp = a.ws + p.off_p + v0 * (3 * 8 * kFrag);
    const T* gp = (const T*)a.dout + row1 * ldo + (size_t)at.h * p.dv;
    unsigned ooff[2][4], ocol[NT];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ooff[0][e] = (unsigned)(ra + e) * ldo;
      ooff[1][e] = (unsigned)(rb + e) * ldo;
    }
#pragma unroll
    for (int u = 0; u < NT; ++u) ocol[u] = at.col(u) < p.dv ? at.col(u) : 0;
    auto load = [&](bool whole) {   // by the moving pointers
      ev[0] = *reinterpret_cast<const v4f*>(dp->e + ra);
      ev[1] = *reinterpret_cast<const v4f*>(dp->e + rb);
      if (whole) {
#pragma unroll
        for (int u = 0; u < NT; ++u)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              go[u][t][e] = ((const GLOBAL T*)gp)[ooff[t][e] + ocol[u]];
      } else {   // rows behind the end: Q and P are zero there
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = (t ? rb : ra) + e;
            const unsigned o = (unsigned)(i < last ? i : last - 1) * ldo;
#pragma unroll
            for (int u = 0; u < NT; ++u) go[u][t][e] = ((const GLOBAL T*)gp)[o + ocol[u]];
          }
      }
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        p0[0][q] = load_frag(pp + (size_t)j * 2 * kFrag, q * 8, off);
        p0[1][q] = load_frag(pp + (size_t)j * 2 * kFrag, q * 8 + 1, off);
        p1[q] = load_frag(pp + (size_t)(3 - j) * 2 * kFrag, q * 8 + 1, off);
      }
#pragma unroll
      for (int q = 0; q < PARTS; ++q)
#pragma unroll
        for (int t = 0; t < QT; ++t)
#pragma unroll
          for (int ks = 0; ks < 2; ++ks)
            qa[t][ks][q] = load_frag(qp, (q * (DKP / 16) + t) * 2 + ks, off);
    };
    auto put = [&] {
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          v4f g;
#pragma unroll
          for (int e = 0; e < 4; ++e) g[e] = to_f32(go[u][t][e]);
          put4<PARTS>(ot, g, 16 * u + lr, t ? rb : ra);
          put4<3>(et, g * (ev[t] * a.scale), 16 * u + lr, t ? rb : ra);
        }
    };
    auto product = [&](int b) {
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        const int col = 16 * u + lr;
        v4f g0 = zero, g1 = zero;
        v8bf oa[PARTS], ob[PARTS];
        get8<PARTS>(ot, oa, col, lg * 8);
        get8<PARTS>(ot, ob, col, 32 + lg * 8);
        g0 = mfma_parts<3>(p0[0], oa, g0);
        g1 = mfma_parts<3>(p1, ob, g1);
        g0 = mfma_parts<3>(p0[1], ob, g0);
        *reinterpret_cast<v4f*>(&d1[b][col][ra]) = g0;
        *reinterpret_cast<v4f*>(&d1[b][col][rb]) = g1;
        v4f x[QT];
#pragma unroll
        for (int t = 0; t < QT; ++t) x[t] = zero;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          v8bf eb[3];
          get8<3>(et, eb, col, ks * 32 + lg * 8);
#pragma unroll
          for (int t = 0; t < QT; ++t) x[t] = mfma_parts<3>(qa[t][ks], eb, x[t]);
        }
#pragma unroll
        for (int t = 0; t < QT; ++t) {
          const int rt = j * QT + t;
          *reinterpret_cast<v4f*>(&eq[b][col][32 * (rt >> 1) + 8 * lg + 4 * (rt & 1)]) = x[t];
        }
      }
    };
    auto back = [&](int c) {   // chunk c's operands are used up: the next
      if (c > 0) {
        pp -= (size_t)p.Hv * (3 * 8 * kFrag);
        qp -= kstep;
        gp -= (size_t)kChunk * ldo;
        dp -= p.Hv;
      }
      load(c > 0 || last >= kChunk);
    };
    load(last >= kChunk);
    put();
    __syncthreads();
    product((nc - 1) & 1);
    back(nc - 1);
    __syncthreads();
    for (int c = nc - 1; c >= 0; --c) {
      __syncthreads();
      put();       // chunk c - 1
      __syncthreads();
      product((c + 1) & 1);
      back(c > 0 ? c - 1 : 0);
      __syncthreads();
    }
  } else if (nc > 0) {
    const int j = wave - 6, cols = p.dv - at.col0;
    T* op = a.dv ? (T*)a.dv + row1 * ldo + (size_t)at.h * p.dv + at.col0 : nullptr;
    float* fp = reinterpret_cast<float*>(a.ws + p.off_dv) + (v0 * p.dv + at.col0) * kChunk;
    float* zp = reinterpret_cast<float*>(a.ws + p.off_ds) + (v0 * p.dv + at.col0) * p.dk;
    using A = Ahead<PARTS, DKP, true>;
    A ahead;
    ahead.set(p, a, at, j * 64 + lane);
    auto touch = [&](int c, unsigned (&h)[A::kTouch]) {
      // the last chunk, where partial, is the first to be used: too late to touch
      if (c >= 0) ahead.touch(c, h);
    };
    unsigned held[A::kSets][A::kTouch] = {};
    touch(nc - 2, held[1]);
    touch(nc - 3, held[2]);
    __syncthreads();
    __syncthreads();
    for (int c4 = nc - 1; c4 >= 0; c4 -= A::kSets)
#pragma unroll
      for (int u = 0; u < A::kSets; ++u) {
        const int c = c4 - u;
        if (c >= 0) {
          A::settle(held[(u + 3) % A::kSets]);
          touch(c - 3, held[(u + 3) % A::kSets]);
          __syncthreads();
          store_columns(zp, ss, p.dk, cols, j, lane);
          zp -= (size_t)p.Hv * p.dk * p.dv;
          __syncthreads();
          __syncthreads();
          store_columns(fp, vs, kChunk, cols, j, lane);
          fp -= (size_t)p.Hv * kChunk * p.dv;
          if (op) {
            store_rows(op, ldo, vs, cols, c == nc - 1 ? last : kChunk, j, lane);
            op -= (size_t)kChunk * ldo;
          }
        }
      }
  }
}

namespace {

template <typename T, int PARTS, int DKP, int DS>
void go(const s4dplr_delta_plan* p, const DeltaArgs& a, bool bwd, hipStream_t s) {
  const unsigned heads = (unsigned)(p->sequences * p->Hv);
  const unsigned grid = (heads + 7) / 8 * 8 * ((p->dv + DS - 1) / DS);
  if (bwd) delta_scan_bwd_kernel<T, PARTS, DKP, DS><<<grid, 512, 0, s>>>(*p, a);
  else if (a.saved) delta_scan_kernel<T, PARTS, DKP, true, DS><<<grid, 512, 0, s>>>(*p, a);
  else delta_scan_kernel<T, PARTS, DKP, false, DS><<<grid, 512, 0, s>>>(*p, a);
}

// bf16 at 64 < dk <= 128: while blocks of 16 columns are no more than the 256 CUs, more
// of them at once is what counts; beyond, blocks of 32 columns share the loads of a
// chunk's operands (4 sequences of 4096 tokens, 16 heads of 128 x 128, 512 blocks of 16:
// forward with saving 359 -> 317 us, backward 414 -> 295 us).  At dk <= 64 blocks of 16 columns
// are the faster ones (5003 tokens in 13 sequences, 8 heads of 64 x 128: 46 us, 51 with
// 32).  Three parts and dk > 128 leave no room for 32 columns.  fp16 has it (162 304 bytes of
// LDS, no spills) and would gain by it (the same sizes, whole passes: forward 629 us, 525 with
// 32 columns; backward 1256 and 1097).  fp32 at dk > 128 spills about 160 registers a
// lane, in the loop over the chunks: 64 chunks of 8 heads of 256 x 128 take 574 us, 162 in bf16.
template <typename T, int PARTS>
hipError_t scan(const s4dplr_delta_plan* p, const DeltaArgs& a, bool bwd, hipStream_t s) {
  const long blocks = (long)p->sequences * p->Hv * ((p->dv + 15) / 16);
  if constexpr (PARTS == 1) {
    if (p->dkp == 128 && p->dv > 16 && blocks > 256) {
      go<T, PARTS, 128, 32>(p, a, bwd, s);
      return hipGetLastError();
    }
  }
  if (p->dkp == 64) go<T, PARTS, 64, 16>(p, a, bwd, s);
  else if (p->dkp == 128) go<T, PARTS, 128, 16>(p, a, bwd, s);
  else go<T, PARTS, 256, 16>(p, a, bwd, s);
  return hipGetLastError();
}

hipError_t scan_any(const s4dplr_delta_plan* p, const DeltaArgs& a, bool bwd, hipStream_t s) {
  if (p->dtype == S4DPLR_F32) return scan<float, 3>(p, a, bwd, s);
  if (p->dtype == S4DPLR_BF16) return scan<bf16, 1>(p, a, bwd, s);
  return scan<f16, 2>(p, a, bwd, s);
}

}  // namespace

hipError_t launch_delta_scan(const s4dplr_delta_plan* p, const DeltaArgs& a, hipStream_t s) {
  return scan_any(p, a, false, s);
}
hipError_t launch_delta_scan_bwd(const s4dplr_delta_plan* p, const DeltaArgs& a, hipStream_t s) {
  return scan_any(p, a, true, s);
}

}  // namespace s4
