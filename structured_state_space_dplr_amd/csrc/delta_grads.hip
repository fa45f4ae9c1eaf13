// Gated delta rule, backward, stage 3: the gradients of q, k, beta and g from what
// the two scans left of each chunk (N, S of the forward one; dV, Z of the backward
// one).  One block per chunk and key head, over the value heads of its group, so
// shared heads are summed in a fixed order:
//   Y = dO N^T, W = dV N^T (64 x 64), F = N Z^T, G1 = dO S^T, G2 = dV S^T (64 x dk),
//   dQ = scale e . G1 + A K,            A_ij = scale beta_j Gam_ij Y_ij (i >= j),
//   dK = -e . G2 + d beta . F + A^T Q - (B + B^T) K,  B_ij = beta_j Gam_ij W_ij (i > j),
//   dbeta_j = sum_i (P_ij Y_ij - H_ij W_ij) + d_j k_j . F_j,
//   dg_t = sum_{i >= t > j} x_ij + sum_{i >= t} (scale e_i q_i . G1_i - e_i k_i . G2_i)
//          + sum_{j < t} d_j beta_j k_j . F_j + e_last <S, Z>,
//   x_ij = beta_j (P_ij Y_ij - H_ij W_ij).
// dg by the pairs that straddle t: summing row and column totals instead would
// take small values as differences of large ones.
//
// Bound by memory: N, S, dV and Z are read once, 4 (2 * 64 dv + 2 dk dv) bytes a chunk
// and head.  They are [dv][..] in memory, 32 of dv a step, and go through LDS as bf16
// parts; the products' k index is dv, so operands come out of LDS with the
// transposing read.  8 waves: wave (w, half) has the chunk's row tile w and half of
// the columns.
//
// Bound by memory: N, S, dV and Z are read once, 4 (2 * 64 dv + 2 dk dv) bytes a chunk
// and head.  They are [dv][..] in memory, 32 of dv a step, and go through LDS as bf16
// parts; the products' k index is dv, so operands come out of LDS with the
// transposing read.  8 waves: wave (w, half) has the chunk's row tile w and half of
// the columns.
//
// Bound by memory: N, S, dV and Z are read once, 4 (2 * 64 dv + 2 dk dv) bytes a chunk
// and head.  They are [dv][..] in memory, 32 of dv a step, and go through LDS as bf16
// parts; the products' k index is dv, so operands come out of LDS with the
// transposing read.  8 waves: wave (w, half) has the chunk's row tile w and half of
// the columns.
//
// Bound by memory: N, S, dV and Z are read once, 4 (2 * 64 dv + 2 dk dv) bytes a chunk
// and head.  They are [dv][..] in memory, 32 of dv a step, and go through LDS as bf16
// parts; the products' k index is dv, so operands come out of LDS with the
// transposing read.  8 waves: wave (w, half) has the chunk's row tile w and half of
// the columns.
#include "delta_device.h"

namespace s4 {

namespace {

constexpr int kLd = 68;

// Operand of 16 columns (the fast index of m [32][LD]) by 32 k (its rows): lane
// (lr, lg) gets column lr, rows 8 lg .. + 8.  In the transposing read 16 lanes
// fetch 4 rows of 16 columns and lane i receives column i.
template <int P, int LD>
__device__ __forceinline__ void get_tr(const __bf16 (*m)[32][LD], int c0, int lr, int lg,
                                       v8bf (&out)[P]) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) v4s lds4;
#pragma unroll
  for (int q = 0; q < P; ++q) {
    const __bf16* a = &m[q][8 * lg + (lr >> 2)][c0 + 4 * (lr & 3)];
    union {
      v4s h[2];
      v8bf v;
    } u;
    u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)a);
    u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(a + 4 * LD));
    out[q] = u.v;
  }
}

// A tile of 32 rows (of dv) by COLS of a [dv][cols] fp32 matrix, by 512 threads: 4
// columns at a time, row (thread + 512 i) / (COLS / 4).  Zero outside the matrix.
template <int COLS>
struct Tile {
  static constexpr int N = 32 * COLS / 4 / 512;
  v4f x[N];
  // m: the tile's first row; rows, cols: what is left of the matrix.  Loads outside are
  // led to element 0 and replaced by 0: no branches.
  __device__ __forceinline__ void load(const float* m, int rows, int cols, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = tid + 512 * i, r = at / (COLS / 4), c = at % (COLS / 4) * 4;
      const unsigned o = (unsigned)(r * cols + c);
      if (cols % 4 == 0) {
        const bool in = r < rows && c < cols;
        const v4f t = *reinterpret_cast<const v4f*>(m + (in ? o : 0u));
        x[i] = in ? t : v4f{0.f, 0.f, 0.f, 0.f};
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool in = r < rows && c + e < cols;
          const float t = m[in ? o + e : 0u];
          x[i][e] = in ? t : 0.f;
        }
      }
    }
  }
  template <int LD>
  __device__ __forceinline__ void put(__bf16 (*to)[32][LD], int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = tid + 512 * i, r = at / (COLS / 4), c = at % (COLS / 4) * 4;
      v4bf t[3];
      split4<3>(x[i], t);
#pragma unroll
      for (int q = 0; q < 3; ++q) *reinterpret_cast<v4bf*>(&to[q][r][c]) = t[q];
    }
  }
};

// Four values, the first n of them.
template <typename T>
__device__ __forceinline__ void store4(T* p, int n, v4f x) {
  T t[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) t[e] = from_f32<T>(x[e]);
  if (n >= 4) {
    __builtin_memcpy(p, t, sizeof(t));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) p[e] = t[e];
  }
}

}  // namespace

template <typename T, int PARTS, int OUTS, int DKP>
__global__ __launch_bounds__(512) void delta_grads_kernel(const s4dplr_delta_plan p,
                                                          const DeltaArgs a) {
  constexpr int KS = DKP / 32, CT = DKP / 32;   // k steps of dk; column tiles of one half
  constexpr int LDN = 64 + 16, LDS_ = DKP + 16; // rows 8 banks apart
  struct Stage {
    __bf16 n[3][32][LDN], v[3][32][LDN], s[3][32][LDS_], z[3][32][LDS_];
  };
  struct Pairs {
    float ym[64][kLd], bm[64][kLd], xm[64][kLd];
  };
  union Mem {
    Stage st;
    Pairs pr;
  };
  __shared__ __attribute__((aligned(16))) Mem mem;
  __shared__ float colsum[4][64];                    // dbeta's pair sums by row tile
  __shared__ float qg[2][64], kg[2][64], kfv[2][64], sz[8], eps[64], xs[64];
  const long slot = blockIdx.x;
  const int hk = blockIdx.y, group = p.Hv / p.Hk;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave & 3, half = wave >> 2;
  const int s = sequence_of(p, a.offsets, slot);
  const Rows r = rows_of(p, a.offsets, s);
  const long c = slot - r.first(s);
  if (c < 0 || c * kChunk >= r.len) return;
  const long t0 = r.start + c * kChunk;
  const int n = (int)(r.len - c * kChunk < kChunk ? r.len - c * kChunk : kChunk);
  const size_t kslot = (size_t)slot * p.Hk + hk;
  constexpr size_t kbytes = (size_t)PARTS * 4 * KS * kFrag;
  const unsigned char* kf = a.ws + p.off_k + kslot * kbytes;
  const unsigned char* qf = a.ws + p.off_q + kslot * kbytes;
  const unsigned char* ktf = a.ws + p.off_kt + kslot * kbytes;
  const unsigned char* qtf = a.ws + p.off_qt + kslot * kbytes;
  const int lr = lane & 15, lg = lane >> 4, i0 = 16 * w + 4 * lg, row = 16 * w + lr;
  const unsigned off = lane * 16;
  const v4f zero = {0.f, 0.f, 0.f, 0.f};

  v4f dq[CT], dk[CT];
#pragma unroll
  for (int i = 0; i < CT; ++i) dq[i] = dk[i] = zero;

  for (int hv = 0; hv < group; ++hv) {
    const int h = hk * group + hv;
    const size_t vslot = (size_t)slot * p.Hv + h;
    const DeltaVec* vec = reinterpret_cast<const DeltaVec*>(a.ws + p.off_vec) + vslot;
    const float* N = reinterpret_cast<const float*>(a.saved + p.off_n) + vslot * kChunk * p.dv;
    const float* S = reinterpret_cast<const float*>(a.saved + p.off_s) + vslot * p.dk * p.dv;
    const float* V = reinterpret_cast<const float*>(a.ws + p.off_dv) + vslot * kChunk * p.dv;
    const float* Z = reinterpret_cast<const float*>(a.ws + p.off_ds) + vslot * p.dk * p.dv;
    const T* go = (const T*)a.dout + ((size_t)(t0 + row) * p.Hv + h) * p.dv;
    const float er = vec->e[row], dbr = vec->d[row] * vec->beta[row];

    // The wave's columns: tiles 2 half, 2 half + 1 of the pair matrices, CT half .. of dk.
    // The products with dk columns are taken transposed: a lane has row `row`, four
    // neighbouring columns.
    v4f y[2], wv[2], f[CT], g1[CT], g2[CT];
#pragma unroll
    for (int i = 0; i < 2; ++i) y[i] = wv[i] = zero;
#pragma unroll
    for (int i = 0; i < CT; ++i) f[i] = g1[i] = g2[i] = zero;
    float dot = 0.f;
    Tile<64> tn, tv;
    Tile<DKP> ts, tz;
    float ox[8];
    auto load = [&](int k0) {
      tn.load(N + (size_t)k0 * 64, p.dv - k0, 64, tid);
      tv.load(V + (size_t)k0 * 64, p.dv - k0, 64, tid);
      ts.load(S + (size_t)k0 * p.dk, p.dv - k0, p.dk, tid);
      tz.load(Z + (size_t)k0 * p.dk, p.dv - k0, p.dk, tid);
      load8(go + k0 + 8 * lg, row < n ? p.dv - k0 - 8 * lg : 0, ox);
    };
    load(0);
    for (int k0 = 0; k0 < p.dv; k0 += 32) {
      __syncthreads();
      tn.put(mem.st.n, tid);
      tv.put(mem.st.v, tid);
      ts.put(mem.st.s, tid);
      tz.put(mem.st.z, tid);
      v8bf oa[PARTS];
      split8<PARTS>(ox, oa);
#pragma unroll
      for (int i = 0; i < Tile<DKP>::N; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) dot = fmaf(ts.x[i][e], tz.x[i][e], dot);
      __syncthreads();
      if (k0 + 32 < p.dv) load(k0 + 32);
      v8bf va[3], na[3], b[3];
      get_tr<3>(mem.st.v, 16 * w, lr, lg, va);
      get_tr<3>(mem.st.n, 16 * w, lr, lg, na);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (2 * half + i <= w) {
          get_tr<3>(mem.st.n, 16 * (2 * half + i), lr, lg, b);
          y[i] = mfma_parts<3>(oa, b, y[i]);
          wv[i] = mfma_parts<3>(va, b, wv[i]);
        }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < CT; ++i) {
        const int c0 = 16 * (CT * half + i);
        get_tr<3>(mem.st.s, c0, lr, lg, b);
        g1[i] = mfma_parts<3>(b, oa, g1[i]);
        g2[i] = mfma_parts<3>(b, va, g2[i]);
        get_tr<3>(mem.st.z, c0, lr, lg, b);
        f[i] = mfma_parts<3>(b, na, f[i]);
        __builtin_amdgcn_sched_barrier(0);   // else all tiles' reads are live at once
      }
    }
    dot = sum64(dot);
    if (lane == 0) sz[wave] = dot;
    __builtin_amdgcn_sched_barrier(0);
    // the operands of row tile w of Q and K: also the rows' elements in the order of
    // the transposed accumulators
    v8bf qa[KS][PARTS], ka[KS][PARTS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int q = 0; q < PARTS; ++q) {
        qa[ks][q] = load_frag(qf + (size_t)w * KS * kFrag, q * 4 * KS + ks, off);
        ka[ks][q] = load_frag(kf + (size_t)w * KS * kFrag, q * 4 * KS + ks, off);
      }
    // rows' products with q and k
    {
      float a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
      for (int i = 0; i < CT; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // k step of column tile CT half + i; a half is whole steps, or (DKP = 64) one
          const int ks = i >> 1, en = 4 * (i & 1) + e;
          float qv = 0.f, kv = 0.f;
#pragma unroll
          for (int q = PARTS - 1; q >= 0; --q) {
            qv += (float)(half ? qa[KS / 2 + ks][q][en] : qa[ks][q][en]);
            kv += (float)(half ? ka[KS / 2 + ks][q][en] : ka[ks][q][en]);
          }
          a1 = fmaf(qv, g1[i][e], a1);
          a2 = fmaf(kv, g2[i][e], a2);
          a3 = fmaf(kv, f[i][e], a3);
        }
        dq[i] += g1[i] * (er * a.scale);
        dk[i] += f[i] * dbr - g2[i] * er;
      }
      a1 += __shfl_xor(a1, 16);
      a2 += __shfl_xor(a2, 16);
      a3 += __shfl_xor(a3, 16);
      a1 += __shfl_xor(a1, 32);
      a2 += __shfl_xor(a2, 32);
      a3 += __shfl_xor(a3, 32);
      if (lg == 0) {
        qg[half][row] = a1;
        kg[half][row] = a2;
        kfv[half][row] = a3;
      }
    }
    __syncthreads();   // the stage's memory becomes the pair matrices'
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int ct = 2 * half + i, j = 16 * ct + lr;
      v4f pp = zero, hh = zero;
      if (ct <= w) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          v8bf kb[PARTS];
#pragma unroll
          for (int q = 0; q < PARTS; ++q)
            kb[q] = load_frag(kf + (size_t)ct * KS * kFrag, q * 4 * KS + ks, off);
          pp = mfma_parts<3>(qa[ks], kb, pp);
          hh = mfma_parts<3>(ka[ks], kb, hh);
        }
      }
      const float bj = vec->beta[j];
      const double Gj = vec->G[j];
      float cs = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int q = i0 + e;
        const float gam = q >= j ? exp_diff(vec->G[q] - Gj) : 0.f;
        const float py = q >= j ? a.scale * gam * pp[e] * y[i][e] : 0.f;
        const float hw = q > j ? gam * hh[e] * wv[i][e] : 0.f;
        cs += py - hw;
        mem.pr.ym[q][j] = q >= j ? a.scale * bj * gam * y[i][e] : 0.f;
        mem.pr.bm[q][j] = q > j ? bj * gam * wv[i][e] : 0.f;
        mem.pr.xm[q][j] = q > j ? bj * (py - hw) : 0.f;
      }
      cs += __shfl_xor(cs, 16);
      cs += __shfl_xor(cs, 32);
      if (lg == 0) colsum[w][j] = cs;
    }
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    // dQ += A K, dK += A^T Q - (B + B^T) K
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const int j0 = ks * 32 + lg * 8;
      float x[8];
      v8bf ya[OUTS], yt[OUTS], ba[OUTS];
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = mem.pr.ym[row][j0 + q];
      split8<OUTS>(x, ya);
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = mem.pr.ym[j0 + q][row];
      split8<OUTS>(x, yt);
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = -(mem.pr.bm[row][j0 + q] + mem.pr.bm[j0 + q][row]);
      split8<OUTS>(x, ba);
#pragma unroll
      for (int i = 0; i < CT; ++i) {
        v8bf kb[PARTS], qb[PARTS];
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
          const int at = q * (DKP / 16) * 2 + i * 2 + ks;
          kb[q] = load_frag(ktf + half * (CT * 2 * kFrag), at, off);
          qb[q] = load_frag(qtf + half * (CT * 2 * kFrag), at, off);
        }
        dq[i] = mfma_parts<3>(kb, ya, dq[i]);
        dk[i] = mfma_parts<3>(qb, yt, dk[i]);
        dk[i] = mfma_parts<3>(kb, ba, dk[i]);
        if (i & 1) __builtin_amdgcn_sched_barrier(0);
      }
    }
    // dbeta, dg
    if (tid < 64) {
      eps[tid] = vec->e[tid] * (a.scale * (qg[0][tid] + qg[1][tid]) - (kg[0][tid] + kg[1][tid]));
      xs[tid] = vec->d[tid] * vec->beta[tid] * (kfv[0][tid] + kfv[1][tid]);
      // xm[i][t] becomes sum_{j < t} x_ij
      float run = 0.f;
#pragma unroll 16
      for (int j = 0; j < 64; ++j) {
        const float t = mem.pr.xm[tid][j];
        mem.pr.xm[tid][j] = run;
        run += t;
      }
    }
    __syncthreads();
    if (tid < 64) {
      const int t = tid;
      float u = 0.f;
#pragma unroll 16
      for (int i = 63; i >= 0; --i) u += i >= t ? mem.pr.xm[i][t] + eps[i] : xs[i];
      const float ss = ((sz[0] + sz[1]) + (sz[2] + sz[3])) + ((sz[4] + sz[5]) + (sz[6] + sz[7]));
      if (t < n) {
        const size_t at = (size_t)(t0 + t) * p.Hv + h;
        if (a.dg) a.dg[at] = u + vec->e[kChunk - 1] * ss;
        if (a.dbeta)
          a.dbeta[at] = ((colsum[0][t] + colsum[1][t]) + (colsum[2][t] + colsum[3][t])) +
                        vec->d[t] * (kfv[0][t] + kfv[1][t]);
      }
    }
    __syncthreads();
  }
  if (row >= n) return;
  const size_t to = ((size_t)(t0 + row) * p.Hk + hk) * p.dk;
#pragma unroll
  for (int i = 0; i < CT; ++i) {
    const int d = 16 * (CT * half + i) + 4 * lg;
    if (a.dq) store4((T*)a.dq + to + d, p.dk - d, dq[i]);
    if (a.dk) store4((T*)a.dk + to + d, p.dk - d, dk[i]);
  }
}

namespace {

template <typename T, int PARTS, int OUTS>
hipError_t grads(const s4dplr_delta_plan* p, const DeltaArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)p->slots, (unsigned)p->Hk);
  if (p->dkp == 64) delta_grads_kernel<T, PARTS, OUTS, 64><<<grid, 512, 0, s>>>(*p, a);
  else if (p->dkp == 128) delta_grads_kernel<T, PARTS, OUTS, 128><<<grid, 512, 0, s>>>(*p, a);
  else delta_grads_kernel<T, PARTS, OUTS, 256><<<grid, 512, 0, s>>>(*p, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_grads(const s4dplr_delta_plan* p, const DeltaArgs& a, hipStream_t s) {
  if (p->dtype == S4DPLR_F32) return grads<float, 3, 3>(p, a, s);
  if (p->dtype == S4DPLR_BF16) return grads<bf16, 1, 2>(p, a, s);
  return grads<f16, 2, 2>(p, a, s);
}

}  // namespace s4
