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
#include "delta_device.h"

namespace s4 {

namespace {
constexpr int kLd = 68;
}

template <typename T, int PARTS, int OUTS, int DKP>
__global__ __launch_bounds__(256) void delta_grads_kernel(const s4dplr_delta_plan p,
                                                          const DeltaArgs a) {
  constexpr int KS = DKP / 32, CT = DKP / 16;
  __shared__ float ym[64][kLd], bm[64][kLd], xm[64][kLd];
  __shared__ float colsum[4][64];                    // dbeta's pair sums by wave
  __shared__ float qg[64], kg[64], kfv[64], sz[4], eps_[64], xs[64];
  const long slot = blockIdx.x;
  const int hk = blockIdx.y, group = p.Hv / p.Hk;
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int s = sequence_of(a.offsets, p.tokens, p.sequences, slot);
  const Rows r = rows_of(a.offsets, p.tokens, p.sequences, s);
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
    const T* go = (const T*)a.dout + ((size_t)t0 * p.Hv + h) * p.dv;
    const size_t ldo = (size_t)p.Hv * p.dv;
    const v4f ev = *reinterpret_cast<const v4f*>(vec->e + i0);
    const v4f dv = *reinterpret_cast<const v4f*>(vec->d + i0);
    const v4f bv = *reinterpret_cast<const v4f*>(vec->beta + i0);

    v4f y[4], wv[4], f[CT], g1[CT], g2[CT];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = wv[i] = zero;
#pragma unroll
    for (int i = 0; i < CT; ++i) f[i] = g1[i] = g2[i] = zero;
    for (int k0 = 8 * lg; k0 - 8 * lg < p.dv; k0 += 32) {
      float x[8];
      v8bf oa[PARTS], va[3], na[3];
      load8(go + (size_t)row * ldo + k0, row < n ? p.dv - k0 : 0, x);
      split8<PARTS>(x, oa);
      load8(V + (size_t)row * p.dv + k0, p.dv - k0, x);
      split8<3>(x, va);
      load8(N + (size_t)row * p.dv + k0, p.dv - k0, x);
      split8<3>(x, na);
#pragma unroll
      for (int ct = 0; ct < 4; ++ct)
        if (ct <= w) {
          v8bf nb[3];
          load8(N + (size_t)(16 * ct + lr) * p.dv + k0, p.dv - k0, x);
          split8<3>(x, nb);
          y[ct] = mfma_parts<3>(oa, nb, y[ct]);
          wv[ct] = mfma_parts<3>(va, nb, wv[ct]);
        }
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const int d = 16 * ct + lr;
        v8bf sb[3];
        load8(S + (size_t)d * p.dv + k0, d < p.dk ? p.dv - k0 : 0, x);
        split8<3>(x, sb);
        g1[ct] = mfma_parts<3>(oa, sb, g1[ct]);
        g2[ct] = mfma_parts<3>(va, sb, g2[ct]);
        load8(Z + (size_t)d * p.dv + k0, d < p.dk ? p.dv - k0 : 0, x);
        split8<3>(x, sb);
        f[ct] = mfma_parts<3>(na, sb, f[ct]);
      }
    }
    // <S, Z>
    float dot = 0.f;
    for (int i = tid; i < p.dk * p.dv; i += 256) dot = fmaf(S[i], Z[i], dot);
    dot = sum64(dot);
    if (lane == 0) sz[w] = dot;
    // rows' products with q and k
    {
      v4f a1 = zero, a2 = zero, a3 = zero;
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const int d = 16 * ct + lr;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool on = i0 + e < n && d < p.dk;
          const float qv =
              on ? to_f32(((const T*)a.q)[(t0 + i0 + e) * a.ldq + (size_t)hk * p.dk + d]) : 0.f;
          const float kv =
              on ? to_f32(((const T*)a.k)[(t0 + i0 + e) * a.ldk + (size_t)hk * p.dk + d]) : 0.f;
          a1[e] = fmaf(qv, g1[ct][e], a1[e]);
          a2[e] = fmaf(kv, g2[ct][e], a2[e]);
          a3[e] = fmaf(kv, f[ct][e], a3[e]);
        }
        dq[ct] += g1[ct] * (ev * a.scale);
        dk[ct] += f[ct] * (dv * bv) - g2[ct] * ev;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float b1 = sum16(a1[e]), b2 = sum16(a2[e]), b3 = sum16(a3[e]);
        if (lr == 0) {
          qg[i0 + e] = b1;
          kg[i0 + e] = b2;
          kfv[i0 + e] = b3;
        }
      }
    }
    // the pair matrices
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) {
      const int j = 16 * ct + lr;
      v4f pp = zero, hh = zero;
      if (ct <= w) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          v8bf qa[PARTS], ka[PARTS], kb[PARTS];
#pragma unroll
          for (int q = 0; q < PARTS; ++q) {
            qa[q] = load_frag(qf, (q * 4 + w) * KS + ks, lane);
            ka[q] = load_frag(kf, (q * 4 + w) * KS + ks, lane);
            kb[q] = load_frag(kf, (q * 4 + ct) * KS + ks, lane);
          }
          pp = mfma_parts<3>(qa, kb, pp);
          hh = mfma_parts<3>(ka, kb, hh);
        }
      }
      const float bj = vec->beta[j];
      const double Gj = vec->G[j];
      float cs = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + e;
        const float gam = i >= j ? exp_diff(vec->G[i] - Gj) : 0.f;
        const float py = i >= j ? a.scale * gam * pp[e] * y[ct][e] : 0.f;
        const float hw = i > j ? gam * hh[e] * wv[ct][e] : 0.f;
        cs += py - hw;
        ym[i][j] = i >= j ? a.scale * bj * gam * y[ct][e] : 0.f;
        bm[i][j] = i > j ? bj * gam * wv[ct][e] : 0.f;
        xm[i][j] = i > j ? bj * (py - hw) : 0.f;
      }
      cs += __shfl_xor(cs, 16);
      cs += __shfl_xor(cs, 32);
      if (lg == 0) colsum[w][j] = cs;
    }
    __syncthreads();
    // dQ += A K, dK += A^T Q - (B + B^T) K
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const int j0 = ks * 32 + lg * 8;
      float x[8];
      v8bf ya[OUTS], yt[OUTS], ba[OUTS];
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = ym[row][j0 + q];
      split8<OUTS>(x, ya);
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = ym[j0 + q][row];
      split8<OUTS>(x, yt);
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = -(bm[row][j0 + q] + bm[j0 + q][row]);
      split8<OUTS>(x, ba);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        v8bf kb[PARTS], qb[PARTS];
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
          kb[q] = load_frag(ktf, (q * CT + ct) * 2 + ks, lane);
          qb[q] = load_frag(qtf, (q * CT + ct) * 2 + ks, lane);
        }
        dq[ct] = mfma_parts<3>(ya, kb, dq[ct]);
        dk[ct] = mfma_parts<3>(yt, qb, dk[ct]);
        dk[ct] = mfma_parts<3>(ba, kb, dk[ct]);
      }
    }
    // dbeta, dg
    if (tid < 64) {
      eps_[tid] = vec->e[tid] * (a.scale * qg[tid] - kg[tid]);
      xs[tid] = vec->d[tid] * vec->beta[tid] * kfv[tid];
      // prefix sums over j of row tid: xm[i][t] becomes sum_{j < t} x_ij
      float run = 0.f;
      for (int j = 0; j < 64; ++j) {
        const float t = xm[tid][j];
        xm[tid][j] = run;
        run += t;
      }
    }
    __syncthreads();
    if (tid < 64) {
      const int t = tid;
      float u = 0.f;
      for (int i = 63; i >= 0; --i)
        u += i >= t ? xm[i][t] + eps_[i] : xs[i];
      const float ss = (sz[0] + sz[1]) + (sz[2] + sz[3]);
      if (t < n) {
        const size_t at = (size_t)(t0 + t) * p.Hv + h;
        if (a.dg) a.dg[at] = u + vec->e[kChunk - 1] * ss;
        if (a.dbeta)
          a.dbeta[at] = ((colsum[0][t] + colsum[1][t]) + (colsum[2][t] + colsum[3][t])) +
                        vec->d[t] * kfv[t];
      }
    }
    __syncthreads();
  }
  // the products' column is a k column, the rows are tokens
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int d = 16 * ct + lr;
    if (d < p.dk)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i0 + e < n) {
          const size_t at = ((size_t)(t0 + i0 + e) * p.Hk + hk) * p.dk + d;
          if (a.dq) ((T*)a.dq)[at] = from_f32<T>(dq[ct][e]);
          if (a.dk) ((T*)a.dk)[at] = from_f32<T>(dk[ct][e]);
        }
  }
}

namespace {

template <typename T, int PARTS, int OUTS>
hipError_t grads(const s4dplr_delta_plan* p, const DeltaArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)p->slots, (unsigned)p->Hk);
  if (p->dkp == 64) delta_grads_kernel<T, PARTS, OUTS, 64><<<grid, 256, 0, s>>>(*p, a);
  else if (p->dkp == 128) delta_grads_kernel<T, PARTS, OUTS, 128><<<grid, 256, 0, s>>>(*p, a);
  else delta_grads_kernel<T, PARTS, OUTS, 256><<<grid, 256, 0, s>>>(*p, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_grads(const s4dplr_delta_plan* p, const DeltaArgs& a, hipStream_t s) {
  if (p->dtype == S4DPLR_F32) return grads<float, 3, 3>(p, a, s);
  if (p->dtype == S4DPLR_BF16) return grads<bf16, 1, 2>(p, a, s);
  return grads<f16, 2, 2>(p, a, s);
}

}  // namespace s4
