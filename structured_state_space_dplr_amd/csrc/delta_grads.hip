// Gated delta rule, backward, stage 3: the gradients of q, k, beta and g from what
// the two scans left of each chunk (N, S of the forward one; dV, Z of the backward
// one):
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
// A block has one chunk, one key head and 64 columns of dk, and walks over the value
// heads of the group, so shared heads are summed in a fixed order.  dg and dbeta are
// linear in the columns: each block writes its part, and delta_gates_kernel adds the
// parts (dk <= 64: there is one, and it is the result).  Blocks of 64 columns keep a
// wave under 256 registers and a block under 50 KB of LDS: two or three share a CU
// and one computes while another loads.  (At 4096 chunks and heads of 128 x 128: 438 us,
// 1.1 GB read; a block for all 128 columns, one to a CU, took 790.)  It waits for loads and
// for LDS: of the CUs' busy time the matrix units take 23 %, vector instructions 36 % and LDS
// 38 %, over half of that for bank conflicts.  fp32 and fp16 at dk > 128 spill (fp32 243
// registers a lane, 341 with grouped heads; fp16 9 and 95).
//
// N, S, dV and Z are [dv][..] in memory, 32 of dv a step, and go through LDS as bf16
// parts; the products' k index is dv, so operands come out of LDS with the
// transposing read.  Wave w has the chunk's row tile w.
#include "delta_device.h"

namespace s4 {

namespace {

constexpr int kLd = 68;
// bf16 from row to row of a staged tile: rows follow one another by 40 banks, so rows 8 apart
// share theirs and the transposing read of 8-column steps meets 8 words on one bank.
constexpr int kLdS = 64 + 16;
constexpr int kCols = 64;       // columns of dk of a block

// A tile of 32 rows (of dv) by 64 columns of an fp32 matrix, by 256 threads: 4 columns
// at a time, rows thread / 16 and + 16.
struct Tile {
  v4f x[2];
  // m: the tile's first element; rows, cols: what is left of the matrix.  Loads outside
  // are led to element 0 and replaced by 0: no branches.
  __device__ __forceinline__ void load(const float* m, int ld, int rows, int cols, int tid) {
    if (rows >= 32 && cols >= 64 && ld % 4 == 0) {   // a whole tile, uniformly
      const unsigned o = (unsigned)((tid >> 4) * ld + (tid & 15) * 4);
      x[0] = *reinterpret_cast<const v4f*>(m + o);
      x[1] = *reinterpret_cast<const v4f*>(m + 16 * (size_t)ld + o);
      return;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = (tid >> 4) + 16 * i, c = (tid & 15) * 4;
      const unsigned o = (unsigned)(r * ld + c);
      if (ld % 4 == 0) {   // then whole groups of 4 are inside or outside
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
  __device__ __forceinline__ void put(__bf16 (*to)[32][kLdS], int tid) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v4bf t[3];
      split4<3>(x[i], t);
#pragma unroll
      for (int q = 0; q < 3; ++q)
        *reinterpret_cast<v4bf*>(&to[q][(tid >> 4) + 16 * i][(tid & 15) * 4]) = t[q];
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

// Three blocks a CU where 168 registers a lane nearly do (9 and 14 are spilled): bf16, one
// value head a key head (no sums over heads are held), and each step's tiles loaded
// when it begins, since the other blocks compute meanwhile (485 -> 428 us at 4096 chunks
// and heads of 128 x 128).  Elsewhere two blocks, with the next step's tiles on their way.
constexpr bool three_blocks(int parts, int dkp, bool grouped) {
  return parts == 1 && dkp <= 128 && !grouped;
}

template <typename T, int PARTS, int DKP, bool GROUPED>
__global__ __launch_bounds__(256, three_blocks(PARTS, DKP, GROUPED) ? 3 : 2) void delta_grads_kernel(const s4dplr_delta_plan p,
                                                             const DeltaArgs a) {
  constexpr int CT = kCols / 16, KS = DKP / 32;
  constexpr bool kThree = three_blocks(PARTS, DKP, GROUPED);
  struct Stage {
    __bf16 v[3][32][kLdS], n[3][32][kLdS], s[3][32][kLdS];
  };
  struct Pairs {
    float ym[64][kLd], bm[64][kLd];
  };
  union Mem {
    Stage st;
    Pairs pr;
  };
  __shared__ __attribute__((aligned(16))) Mem mem;
  __shared__ float colsum[4][64];                    // dbeta's pair sums by row tile
  __shared__ float cross[4][64];                     // dg's, of the pairs i >= t > j
  __shared__ float qg[64], kfv[64], sz[4], xs[64];
  const int nb = (p.dk + kCols - 1) / kCols;
  // the column blocks of a chunk, which share N and dV, on one XCD
  const int slot = (int)(blockIdx.x / (8 * nb)) * 8 + (blockIdx.x & 7), cb = blockIdx.x / 8 % nb;
  if (slot >= p.slots) return;
  const int hk = blockIdx.y, group = GROUPED ? p.Hv / p.Hk : 1;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int s = sequence_of(p, a, slot);
  const Rows r = rows_of(p, a.offsets, s);
  const long c = slot - r.first(s, a.least);
  if (c < 0 || c * kChunk >= r.len) return;
  const long t0 = r.start + c * kChunk;
  const int n = (int)(r.len - c * kChunk < kChunk ? r.len - c * kChunk : kChunk);
  const int c0 = cb * kCols, dcols = p.dk - c0;
  const size_t kbase = ((size_t)slot * p.Hk + hk) * PARTS * 4 * KS * kFrag;
  const unsigned char* kf = a.ws + p.off_k + kbase;
  const unsigned char* qf = a.ws + p.off_q + kbase;
  const unsigned char* ktf = a.ws + p.off_kt + kbase + (size_t)cb * (CT * 2 * kFrag);
  const unsigned char* qtf = a.ws + p.off_qt + kbase + (size_t)cb * (CT * 2 * kFrag);
  const v4f zero = {0.f, 0.f, 0.f, 0.f};

  v4f dq[CT], dk[CT];
#pragma unroll
  for (int i = 0; i < CT; ++i) dq[i] = dk[i] = zero;

  for (int hv = 0; hv < group; ++hv) {
    // opaque: the addresses that follow from it are formed in the loop, where else
    // all of them would be formed ahead of it and spilled
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63;
    const int lr = lane & 15, lg = lane >> 4, i0 = 16 * w + 4 * lg, row = 16 * w + lr;
    const unsigned off = lane * 16;
    const int h = hk * group + hv;
    const size_t vslot = (size_t)slot * p.Hv + h;
    const DeltaVec* vec = reinterpret_cast<const DeltaVec*>(a.ws + p.off_vec) + vslot;
    const float* N = reinterpret_cast<const float*>(a.saved + p.off_n) + vslot * kChunk * p.dv;
    const float* S = reinterpret_cast<const float*>(a.saved + p.off_s) + vslot * p.dk * p.dv + c0;
    const float* V = reinterpret_cast<const float*>(a.ws + p.off_dv) + vslot * kChunk * p.dv;
    const float* Z = reinterpret_cast<const float*>(a.ws + p.off_ds) + vslot * p.dk * p.dv + c0;
    const T* go = (const T*)a.dout + ((size_t)(t0 + row) * p.Hv + h) * p.dv;
    const float er = vec->e[row], dbr = vec->d[row] * vec->beta[row];

    // The products with dk columns are taken transposed: a lane has row `row`, four
    // neighbouring columns of each tile.  Rows behind the end have dO = dV = 0 and
    // beta = 0, columns behind dk are 0.
    v4f y[4], wv[4], g1[CT], g2[CT], f[CT];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = wv[i] = zero;
#pragma unroll
    for (int i = 0; i < CT; ++i) g1[i] = g2[i] = f[i] = zero;
    float dot = 0.f;   // <S, Z>
    Tile tv, tn, ts, tz;
    float ox[8];
    auto load = [&](int k0) {
      tv.load(V + (size_t)k0 * 64, 64, p.dv - k0, 64, tid);
      tn.load(N + (size_t)k0 * 64, 64, p.dv - k0, 64, tid);
      ts.load(S + (size_t)k0 * p.dk, p.dk, p.dv - k0, dcols, tid);
      tz.load(Z + (size_t)k0 * p.dk, p.dk, p.dv - k0, dcols, tid);
      load8(go + k0 + 8 * lg, row < n ? p.dv - k0 - 8 * lg : 0, ox);
    };
    if constexpr (!kThree) load(0);
    for (int k0 = 0; k0 < p.dv; k0 += 32) {
      if constexpr (kThree) load(k0);
      __syncthreads();
      tv.put(mem.st.v, tid);
      tn.put(mem.st.n, tid);
      ts.put(mem.st.s, tid);
      v8bf oa[PARTS], va[3], na[3], b[3];
      split8<PARTS>(ox, oa);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) dot = fmaf(ts.x[i][e], tz.x[i][e], dot);
      const Tile zn = tz;
      __syncthreads();
      if (!kThree && k0 + 32 < p.dv) load(k0 + 32);
      get_tr<3, 4>(mem.st.v, 0, 16 * w, lr, lg, va);
#pragma unroll
      for (int i = 0; i < CT; ++i) {
        get_tr<3, 8>(mem.st.s, 0, 32 * (i >> 1) + 4 * (i & 1), lr, lg, b);
        g1[i] = mfma_parts<3>(b, oa, g1[i]);
        g2[i] = mfma_parts<3>(b, va, g2[i]);
      }
      get_tr<3, 4>(mem.st.n, 0, 16 * w, lr, lg, na);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i <= w) {
          get_tr<3, 4>(mem.st.n, 0, 16 * i, lr, lg, b);
          y[i] = mfma_parts<3>(oa, b, y[i]);
          wv[i] = mfma_parts<3>(va, b, wv[i]);
        }
      __syncthreads();
      zn.put(mem.st.s, tid);   // Z takes S's place
      __syncthreads();
#pragma unroll
      for (int i = 0; i < CT; ++i) {
        get_tr<3, 8>(mem.st.s, 0, 32 * (i >> 1) + 4 * (i & 1), lr, lg, b);
        f[i] = mfma_parts<3>(b, na, f[i]);
      }
    }
    dot = sum64(dot);
    if (lane == 0) sz[w] = dot;
    // Q's and K's operands of row tile w; those of the block's columns are the rows'
    // elements in the order of the accumulators as well
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
      for (int b = 0; b < KS / 2; ++b)
        if (b == cb)
#pragma unroll
          for (int i = 0; i < CT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float q = 0.f, k = 0.f;
#pragma unroll
              for (int j = PARTS - 1; j >= 0; --j) {
                q += (float)qa[2 * b + i / 2][j][4 * (i & 1) + e];
                k += (float)ka[2 * b + i / 2][j][4 * (i & 1) + e];
              }
              a1 = fmaf(q, g1[i][e], a1);
              a2 = fmaf(k, g2[i][e], a2);
              a3 = fmaf(k, f[i][e], a3);
            }
#pragma unroll
      for (int i = 0; i < CT; ++i) {
        const v4f x = g1[i] * (er * a.scale), z = f[i] * dbr - g2[i] * er;
        dq[i] = GROUPED ? dq[i] + x : x;
        dk[i] = GROUPED ? dk[i] + z : z;
      }
      a1 = er * (a.scale * a1 - a2);
      a1 += __shfl_xor(a1, 16);
      a3 += __shfl_xor(a3, 16);
      a1 += __shfl_xor(a1, 32);
      a3 += __shfl_xor(a3, 32);
      if (lg == 0) {
        qg[row] = a1;
        kfv[row] = vec->d[row] * a3;
        xs[row] = dbr * a3;
      }
    }
    // P and H: the pair sums are the first block's
    v4f pp[4], hh[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) pp[i] = hh[i] = zero;
    if (cb == 0)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          v8bf kb[PARTS];
#pragma unroll
          for (int q = 0; q < PARTS; ++q) kb[q] = load_frag(kf, (q * 4 + i) * KS + ks, off);
          pp[i] = mfma_parts<3>(qa[ks], kb, pp[i]);
          hh[i] = mfma_parts<3>(ka[ks], kb, hh[i]);
        }
    // the last products' operands, ahead of what they wait for
    constexpr bool kAhead = PARTS == 1 && !kThree;
    v8bf kc[2][CT][PARTS], qc[2][CT][PARTS];
    auto load_kq = [&](int ks) {
#pragma unroll
      for (int i = 0; i < CT; ++i)
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
          kc[ks][i][q] = load_frag(ktf, q * (DKP / 16) * 2 + i * 2 + ks, off);
          qc[ks][i][q] = load_frag(qtf, q * (DKP / 16) * 2 + i * 2 + ks, off);
        }
    };
    if constexpr (kAhead) {
      load_kq(0);
      load_kq(1);
    }
    __syncthreads();   // the stage's memory becomes the pair matrices'
    double Gi[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) Gi[e] = vec->G[i0 + e];
    // sum_{j < t} x_ij of the lane's rows up to the tile at hand
    float run[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = 16 * i + lr;
      float cs = 0.f, cr = 0.f;
      if (i <= w) {
        const float bj = vec->beta[j];
        const double Gj = vec->G[j];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int q = i0 + e;
          const bool low = q > j, diag = q >= j;
          const float gam = exp_diff(diag ? Gi[e] - Gj : 0.0);
          const float gy = diag ? a.scale * gam * y[i][e] : 0.f;
          const float gw = low ? gam * wv[i][e] : 0.f;
          const float t = gy * pp[i][e] - gw * hh[i][e];
          cs += t;
          mem.pr.ym[q][j] = bj * gy;
          mem.pr.bm[q][j] = bj * gw;
          // sums over the columns up to each, by the 16 lanes of a row of the tile
          float x = low ? bj * t : 0.f;
          x += dpp<0x111>(x);   // row_shr 1, 2, 4, 8
          x += dpp<0x112>(x);
          x += dpp<0x114>(x);
          x += dpp<0x118>(x);
          const float before = run[e] + dpp<0x111>(x);   // columns below j = t
          cr += diag ? before : 0.f;
          run[e] += dpp<0x15F>(x);                       // row_newbcast 15: the tile's sum
        }
        cs += __shfl_xor(cs, 16);
        cr += __shfl_xor(cr, 16);
        cs += __shfl_xor(cs, 32);
        cr += __shfl_xor(cr, 32);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) mem.pr.ym[i0 + e][j] = mem.pr.bm[i0 + e][j] = 0.f;
      }
      if (lg == 0) {
        colsum[w][j] = cs;
        cross[w][j] = cr;
      }
    }
    __syncthreads();
    // dQ += A K, dK += A^T Q - (B + B^T) K
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      if constexpr (!kAhead) load_kq(ks);
      const int j0 = ks * 32 + lg * 8;
      float x[8];
      v8bf ya[3], yt[3], ba[3];
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = mem.pr.ym[row][j0 + q];
      split8<3>(x, ya);
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = mem.pr.ym[j0 + q][row];
      split8<3>(x, yt);
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = -(mem.pr.bm[row][j0 + q] + mem.pr.bm[j0 + q][row]);
      split8<3>(x, ba);
#pragma unroll
      for (int i = 0; i < CT; ++i) {
        dq[i] = mfma_parts<3>(kc[ks][i], ya, dq[i]);
        dk[i] = mfma_parts<3>(qc[ks][i], yt, dk[i]);
        dk[i] = mfma_parts<3>(kc[ks][i], ba, dk[i]);
      }
    }
    // dbeta, dg: token t = lane
    if (w == 0) {
      const int t = tid;
      float after = qg[t], before = xs[t];   // sums over i >= t and, then, j < t
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const float x = __shfl_down(after, off), z = __shfl_up(before, off);
        if (t + off < 64) after += x;
        if (t >= off) before += z;
      }
      before = __shfl_up(before, 1);
      float u = after + (t > 0 ? before : 0.f);
      float cs = 0.f;
      if (cb == 0) {
        u += (cross[0][t] + cross[1][t]) + (cross[2][t] + cross[3][t]);
        cs = (colsum[0][t] + colsum[1][t]) + (colsum[2][t] + colsum[3][t]);
      }
      const float ss = (sz[0] + sz[1]) + (sz[2] + sz[3]);
      const size_t at = (size_t)(t0 + t) * p.Hv + h;
      const size_t all = (size_t)p.tokens * p.Hv;
      float* dg = nb == 1 ? a.dg : reinterpret_cast<float*>(a.ws + p.off_gates) + 2 * cb * all;
      float* db = nb == 1 ? a.dbeta : dg + all;
      if (dg && t < n) dg[at] = u + vec->e[kChunk - 1] * ss;
      if (db && t < n) db[at] = cs + kfv[t];
    }
    __syncthreads();
  }
  const int lg = (threadIdx.x & 63) >> 4, row = 16 * w + (threadIdx.x & 15);
  if (row >= n) return;
  const size_t to = ((size_t)(t0 + row) * p.Hk + hk) * p.dk + c0;
#pragma unroll
  for (int i = 0; i < CT; ++i) {
    const int d = 32 * (i >> 1) + 8 * lg + 4 * (i & 1);
    if (a.dq) store4((T*)a.dq + to + d, dcols - d, dq[i]);
    if (a.dk) store4((T*)a.dk + to + d, dcols - d, dk[i]);
  }
}

// dg and dbeta: the column blocks' parts [block][2][tokens][Hv] added up, over the rows
// that belong to sequences (they follow one another).
__global__ __launch_bounds__(256) void delta_gates_kernel(const s4dplr_delta_plan p,
                                                          const DeltaArgs a) {
  const int nb = (p.dk + kCols - 1) / kCols;
  const size_t all = (size_t)p.tokens * p.Hv;
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  const Rows first = rows_of(p, a.offsets, 0), last = rows_of(p, a.offsets, p.sequences - 1);
  if (i < (size_t)first.start * p.Hv || i >= (size_t)(last.start + last.len) * p.Hv) return;
  const float* part = reinterpret_cast<const float*>(a.ws + p.off_gates);
  float g = 0.f, b = 0.f;
  for (int j = 0; j < nb; ++j) {
    g += part[2 * j * all + i];
    b += part[(2 * j + 1) * all + i];
  }
  if (a.dg) a.dg[i] = g;
  if (a.dbeta) a.dbeta[i] = b;
}

namespace {

template <typename T, int PARTS>
hipError_t grads(const s4dplr_delta_plan* p, const DeltaArgs& a, hipStream_t s) {
  const int nb = (p->dk + kCols - 1) / kCols;
  const dim3 grid((unsigned)((p->slots + 7) / 8 * 8 * nb), (unsigned)p->Hk);
#define S4_GO(dkp)                                                                     \
  (p->Hv > p->Hk ? delta_grads_kernel<T, PARTS, dkp, true><<<grid, 256, 0, s>>>(*p, a) \
                 : delta_grads_kernel<T, PARTS, dkp, false><<<grid, 256, 0, s>>>(*p, a))
  if (p->dkp == 64) S4_GO(64);
  else if (p->dkp == 128) S4_GO(128);
  else S4_GO(256);
#undef S4_GO
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || nb == 1 || p->tokens == 0 || (!a.dg && !a.dbeta)) return e;
  const size_t n = (size_t)p->tokens * p->Hv;
  delta_gates_kernel<<<dim3((unsigned)((n + 255) / 256)), 256, 0, s>>>(*p, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_grads(const s4dplr_delta_plan* p, const DeltaArgs& a, hipStream_t s) {
  if (p->slots == 0) return hipSuccess;   // no tokens
  if (p->dtype == S4DPLR_F32) return grads<float, 3>(p, a, s);
  if (p->dtype == S4DPLR_BF16) return grads<bf16, 1>(p, a, s);
  return grads<f16, 2>(p, a, s);
}

}  // namespace s4
