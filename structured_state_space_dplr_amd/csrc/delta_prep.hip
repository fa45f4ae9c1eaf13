// Gated delta rule, chunked form, stage 1: everything of a chunk that does not
// depend on the state.  One block per chunk and value head:
//   G_i = g_0 + ... + g_i,  Gam_ij = exp(G_i - G_j),
//   H = strictly lower (Gam . K K^T),  P = lower (Gam . Q K^T),
//   X = (I + H diag(beta))^-1,
// written as matrix-instruction operands (with K, Q and K^T, zero-padded), so the
// sequential stage reads them with whole-line loads and no bounds.  The backward
// pass takes X^T, P^T and Q^T instead of X and P.
//
// It is bound by what it reads and writes beside short dependent products (256 chunks of 16
// value heads and 8 key heads of 128 in bf16: 98 us; of 16 key heads 123 us, and 135
// backward, which transposes Q too); 256 threads and 53 KB of LDS let three blocks share a CU, so that
// one writes while another computes.
//
// The inverse is exact fp32: each 16 x 16 diagonal block by forward
// substitution, the blocks below by X_rc = -X_rr sum_m A_rm X_mc with the fp32
// matrix instruction, one wave per block column.
#include "delta_device.h"

namespace s4 {

namespace {

constexpr int kLd = 68;   // floats from row to row of a 64 x 64 matrix in LDS

}  // namespace

template <typename T, int PARTS, int DKP, bool BWD>
__global__ __launch_bounds__(256) void delta_prep_kernel(const s4dplr_delta_plan p,
                                                         const DeltaArgs a) {
  constexpr int KS = DKP / 32;
  __shared__ __attribute__((aligned(16))) __bf16 km[PARTS][64][DKP + 8];   // K, then Q, by rows
  __shared__ float am[64][kLd], pm[64][kLd];
  __shared__ double G[64];
  __shared__ float bt[64];
  const long slot = blockIdx.x;
  const int h = blockIdx.y, hk = h / (p.Hv / p.Hk);
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int s = sequence_of(p, a, slot);
  const Rows r = rows_of(p, a.offsets, s);
  const long c = slot - r.first(s, a.least);
  if (c < 0 || c * kChunk >= r.len || r.len <= a.step_tokens) return;
  const long t0 = r.start + c * kChunk;
  const int n = (int)(r.len - c * kChunk < kChunk ? r.len - c * kChunk : kChunk);
  const bool own_k = h % (p.Hv / p.Hk) == 0;   // one head of a group writes the shared operands
  const size_t kslot = (size_t)slot * p.Hk + hk, vslot = (size_t)slot * p.Hv + h;
  constexpr size_t kbytes = (size_t)PARTS * 4 * KS * kFrag;

  float g0 = 0.f, b0 = 0.f;   // on their way while K and Q are split
  if (w == 0 && lane < n) {
    g0 = a.g[(size_t)(t0 + lane) * p.Hv + h];
    b0 = a.beta[(size_t)(t0 + lane) * p.Hv + h];
  }
  // K and Q of the wave's 16 rows
  const int row = 16 * w + (lane & 15);
  v8bf qr[KS][PARTS];
  {
    const T* kp = (const T*)a.k + (t0 + row) * a.ldk + (size_t)hk * p.dk;
    const T* qp = (const T*)a.q + (t0 + row) * a.ldq + (size_t)hk * p.dk;
    unsigned char* ko = a.ws + p.off_k + kslot * kbytes;
    unsigned char* qo = a.ws + p.off_q + kslot * kbytes;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const int col = ks * 32 + (lane >> 4) * 8;
      const int m = row < n ? p.dk - col : 0;
      float x[8];
      v8bf kk[PARTS];
      load8(kp + col, m, x);
      split8<PARTS>(x, kk);
      load8(qp + col, m, x);
      split8<PARTS>(x, qr[ks]);
#pragma unroll
      for (int i = 0; i < PARTS; ++i) {
        *reinterpret_cast<v8bf*>(&km[i][row][col]) = kk[i];
        if (own_k) {
          const size_t f = ((size_t)(i * 4 + w) * KS + ks) * kFrag + lane * 16;
          *reinterpret_cast<v8bf*>(ko + f) = kk[i];
          *reinterpret_cast<v8bf*>(qo + f) = qr[ks][i];
        }
      }
    }
  }
  // decays: sums in 64 bits, so that a difference keeps its digits behind a
  // large negative g (a reset); below -200 the decay is 0 in fp32 either way
  if (w == 0) {
    DeltaVec* vec = reinterpret_cast<DeltaVec*>(a.ws + p.off_vec) + vslot;
    double x = (g0 < -200.f ? -200.0 : (double)g0) * 1.4426950408889634;   // powers of 2
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const double y = __shfl_up(x, off);
      if (lane >= off) x += y;
    }
    const double last = __shfl(x, 63);
    G[lane] = x;
    bt[lane] = b0;
    vec->e[lane] = exp_diff(x);
    vec->d[lane] = exp_diff(last - x);
    vec->beta[lane] = b0;
    vec->G[lane] = x;
  }
  __syncthreads();

  // H and P, tiles on and below the diagonal; zero elsewhere
#pragma unroll
  for (int ct = 0; ct < 4; ++ct) {
    v4f hh = {0.f, 0.f, 0.f, 0.f}, pp = {0.f, 0.f, 0.f, 0.f};
    if (ct <= w) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        v8bf ka[PARTS], kb[PARTS];
#pragma unroll
        for (int i = 0; i < PARTS; ++i) {
          ka[i] = *reinterpret_cast<const v8bf*>(&km[i][row][ks * 32 + (lane >> 4) * 8]);
          kb[i] = *reinterpret_cast<const v8bf*>(&km[i][16 * ct + (lane & 15)][ks * 32 + (lane >> 4) * 8]);
        }
        hh = mfma_parts<3>(ka, kb, hh);
        pp = mfma_parts<3>(qr[ks], kb, pp);
      }
    }
    const int j = 16 * ct + (lane & 15);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 16 * w + 4 * (lane >> 4) + e;
      const float gam = i >= j ? exp_diff(G[i] - G[j]) : 0.f;
      am[i][j] = i > j ? hh[e] * gam * bt[j] : 0.f;
      pm[i][j] = i >= j ? pp[e] * gam * a.scale : 0.f;
    }
  }
  __syncthreads();

  // X over am: diagonal blocks first
  {
    float x[16];
    const int j = lane & 15, o = 16 * w;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float t = i == j ? 1.f : 0.f;
#pragma unroll
      for (int m = 0; m < 16; ++m)
        if (m < i) t = fmaf(-am[o + i][o + m], x[m], t);
      x[i] = t;
    }
    if (lane < 16)
#pragma unroll
      for (int i = 0; i < 16; ++i) am[o + i][o + j] = x[i];
  }
  __syncthreads();
  // block column w: rows below, from the top; the blocks of A that are read lie in
  // columns that their own wave overwrites, so every wave takes its A first
  {
    const int col = lane & 15, kk = lane >> 4;
    float ab[4][4][4];   // A_rm, r > m >= w
#pragma unroll
    for (int rb = 1; rb < 4; ++rb)
#pragma unroll
      for (int m = 0; m < 3; ++m)
        if (m < rb)
#pragma unroll
          for (int q = 0; q < 4; ++q) ab[rb][m][q] = am[16 * rb + col][16 * m + 4 * q + kk];
    __syncthreads();
#pragma unroll
    for (int rb = 1; rb < 4; ++rb) {
      if (rb <= w) continue;
      v4f t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int m = 0; m < 3; ++m)
        if (m < rb && m >= w)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            t = mfma32(ab[rb][m][q], am[16 * m + 4 * q + kk][16 * w + col], t);
      // the block's place holds t while it is turned into an operand
#pragma unroll
      for (int e = 0; e < 4; ++e) am[16 * rb + 4 * kk + e][16 * w + col] = t[e];
      wave_sync();
      v4f x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        x = mfma32(am[16 * rb + col][16 * rb + 4 * q + kk], am[16 * rb + 4 * q + kk][16 * w + col], x);
      wave_sync();
#pragma unroll
      for (int e = 0; e < 4; ++e) am[16 * rb + 4 * kk + e][16 * w + col] = -x[e];
      wave_sync();
    }
  }
  __syncthreads();

  // operands of X and P (three parts), or of their transposes
  {
    unsigned char* xo = a.ws + p.off_x + vslot * (3 * 8 * kFrag);
    unsigned char* po = a.ws + p.off_p + vslot * (3 * 8 * kFrag);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      if (BWD ? ks < w / 2 : ks > w / 2) continue;   // zero, and never read
      const int k0 = ks * 32 + (lane >> 4) * 8;
      float x[8], y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = BWD ? am[k0 + i][row] : am[row][k0 + i];
        y[i] = BWD ? pm[k0 + i][row] : pm[row][k0 + i];
      }
      v8bf xs[3], ps[3];
      split8<3>(x, xs);
      split8<3>(y, ps);
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const size_t f = (size_t)((i * 4 + w) * 2 + ks) * kFrag + lane * 16;
        *reinterpret_cast<v8bf*>(xo + f) = xs[i];
        *reinterpret_cast<v8bf*>(po + f) = ps[i];
      }
    }
  }
  // K^T (then, through the same memory, Q^T).  Row 4 g + e of tile t of a k step of dk is
  // column 8 g + 4 t + e of the step, so that the two tiles' accumulators hold 8
  // neighbouring rows of the state a lane.
  if (!own_k) return;
#pragma unroll
  for (int pass = 0; pass < (BWD ? 2 : 1); ++pass) {
    unsigned char* to = a.ws + (pass ? p.off_qt : p.off_kt) + kslot * kbytes;
    if (pass) {
      __syncthreads();
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int i = 0; i < PARTS; ++i)
          *reinterpret_cast<v8bf*>(&km[i][row][ks * 32 + (lane >> 4) * 8]) = qr[ks][i];
      __syncthreads();
    }
#pragma unroll
    for (int f = 0; f < DKP / 32; ++f) {   // tiles w, w + 4, ... of DKP / 16, both k steps
      const int at = w + 4 * f, rt = at >> 1, ks = at & 1;
      v8bf t[PARTS];
      get_tr<PARTS, 8>(km, 32 * ks, 32 * (rt >> 1) + 4 * (rt & 1), lane & 15, lane >> 4, t);
#pragma unroll
      for (int q = 0; q < PARTS; ++q)
        *reinterpret_cast<v8bf*>(to + (size_t)((q * (DKP / 16) + rt) * 2 + ks) * kFrag + lane * 16) = t[q];
    }
  }
}

namespace {

template <typename T, int PARTS>
hipError_t prep(const s4dplr_delta_plan* p, const DeltaArgs& a, bool bwd, hipStream_t s) {
  const dim3 grid((unsigned)p->slots, (unsigned)p->Hv);
#define S4_GO(dkp)                                                                     \
  if (bwd)                                                                             \
    delta_prep_kernel<T, PARTS, dkp, true><<<grid, 256, 0, s>>>(*p, a);                \
  else                                                                                 \
    delta_prep_kernel<T, PARTS, dkp, false><<<grid, 256, 0, s>>>(*p, a)
  if (p->dkp == 64) { S4_GO(64); }
  else if (p->dkp == 128) { S4_GO(128); }
  else { S4_GO(256); }
#undef S4_GO
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_prep(const s4dplr_delta_plan* p, const DeltaArgs& a, bool bwd,
                             hipStream_t s) {
  if (p->slots == 0) return hipSuccess;   // no tokens
  if (p->dtype == S4DPLR_F32) return prep<float, 3>(p, a, bwd, s);
  if (p->dtype == S4DPLR_BF16) return prep<bf16, 1>(p, a, bwd, s);
  return prep<f16, 2>(p, a, bwd, s);
}

}  // namespace s4
