// Layer norm, forward and backward, over the middle axis of x [outer][D][inner]:
//   m = mean_d x,  r = 1 / sqrt(mean_d (x - m)^2 + eps),  y = (x - m) r gamma + beta,
//   xh = (x - m) r,  w = dy gamma,
//   dx = r (w - mean_d w - xh mean_d (w xh)),  dgamma = sum dy xh,  dbeta = sum dy.
// inner = 1 is the token-major layout (rows of D contiguous values), inner = L
// the [batch][H][L] layout normalized over its H channels.  Elements are fp32,
// bf16 or fp16; all arithmetic is fp32, each output is rounded once.  The
// variance is the mean of squared deviations from the mean (two passes over
// registers), so a large common offset costs no digits.
//
// Both directions are bound by HBM: forward reads x and writes y, backward reads
// x and dy and writes dx.
#include "norm.h"

#include "vec.h"

namespace s4 {

namespace {

constexpr int kRowThreads = 256;

// A lane's share of a row as it lies in memory: NV vectors, vector i at element
// ((i WPR + wave) 64 + lane) VEC.  WHOLE: D is a multiple of VEC, so a vector is
// inside or outside; one outside is read from the row's start and replaced by 0, with
// no branch for the loads to wait at.
template <typename T, int NV, int WPR, bool WHOLE>
struct RowPart {
  static constexpr int VEC = Vec<T>::N, E = NV * VEC;
  Vec<T> v[NV];
  __device__ __forceinline__ static int at(int i, int tid) { return (i * WPR * 64 + tid) * VEC; }
  __device__ __forceinline__ void load(const T* __restrict__ p, int D, int tid) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = at(i, tid);
      if constexpr (WHOLE) {
        v[i] = load_vec(p + (c < D ? c : 0));
      } else if (c + VEC <= D) {
        v[i] = load_vec(p + c);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i].v[j] = c + j < D ? p[c + j] : (T)0.f;
      }
    }
  }
  __device__ __forceinline__ void get(int D, int tid, float* out) const {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        out[i * VEC + j] = !WHOLE || at(i, tid) < D ? to_f32(v[i].v[j]) : 0.f;
  }
  __device__ __forceinline__ static void store(T* __restrict__ p, int D, int tid, const float* in) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = at(i, tid);
      if (c + VEC <= D) {
        Vec<T> t;
#pragma unroll
        for (int j = 0; j < VEC; ++j) t.v[j] = from_f32<T>(in[i * VEC + j]);
        store_vec(p + c, t);
      } else if constexpr (!WHOLE) {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (c + j < D) p[c + j] = from_f32<T>(in[i * VEC + j]);
      }
    }
  }
  // the same columns of a vector of D floats; `other` where there is none
  __device__ __forceinline__ static void columns(const float* __restrict__ p, int D, int tid,
                                                 float other, float* out) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = at(i, tid);
      if (p && c + VEC <= D) {
        __builtin_memcpy(out + i * VEC, p + c, VEC * sizeof(float));
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) out[i * VEC + j] = p && c + j < D ? p[c + j] : other;
      }
    }
  }
};

// Rows of 32 values a lane: 16 waves have 128 registers a lane, and gamma and beta are
// read where they are used.
constexpr bool wide_rows(int values, int waves) { return waves > 4 && values > 16; }

// The same value, unknown to the compiler: a load at it is not taken out of the loop, where
// its result would be kept in registers and spilled.
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Forward over rows.  WPR waves share a row (blocks of 256 threads hold 4 rows at WPR =
// 1), and a block walks over rows blockIdx, blockIdx + gridDim, ..., the next row on its
// way while one is computed: gamma and beta are read once.  A wave takes mean and
// squared deviations of its own part; the parts are joined by
//   m = sum n_w m_w / D,  M = sum M_w + n_w (m_w - m)^2,
// with one barrier a row (two sets of slots in turn).
template <typename T, int NV, int WPR, bool WHOLE>
__global__ __launch_bounds__(WPR > 4 ? 64 * WPR : kRowThreads) void norm_rows_kernel(
    const T* x, const float* __restrict__ gamma, const float* __restrict__ beta, T* y,
    float* __restrict__ mean, float* __restrict__ rstd, long rows, int D, float eps) {
  using Part = RowPart<T, NV, WPR, WHOLE>;
  constexpr int VEC = Part::VEC, E = Part::E;
  constexpr int RPB = WPR == 1 ? kRowThreads / 64 : 1;
  __shared__ float red[2][2][WPR];
  const int tid = WPR == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  long row = (long)blockIdx.x * RPB + (WPR == 1 ? w : 0);
  if (row >= rows) return;   // WPR > 1: the whole block
  Part next;
  next.load(x + row * D, D, tid);
  constexpr bool kWide = wide_rows(E, WPR);
  float gm[kWide ? 1 : E], bt[kWide ? 1 : E];
  if constexpr (!kWide) {
    Part::columns(gamma, D, tid, 1.f, gm);
    Part::columns(beta, D, tid, 0.f, bt);
  }
  // elements of the wave's part
  float n = (float)D;
  if constexpr (WPR > 1) {
    int c = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int left = D - Part::at(i, 64 * w);
      c += left < 0 ? 0 : left < 64 * VEC ? left : 64 * VEC;
    }
    n = (float)c;
  }
  int turn = 0;
  for (; row < rows; turn ^= 1) {
    float v[E];
    next.get(D, tid, v);
    const long here = row;
    row += (long)gridDim.x * RPB;
    if (row < rows) next.load(x + row * D, D, tid);
    float s = 0.f, q = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s += v[i];
    float m = n > 0.f ? sum64(s) / n : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float d = v[i * VEC + j] - m;
        q += Part::at(i, tid) + j < D ? d * d : 0.f;
      }
    q = sum64(q);
    if constexpr (WPR > 1) {
      if (tid % 64 == 0) {
        red[turn][0][w] = m;
        red[turn][1][w] = q;
      }
      __syncthreads();
      float part[WPR], len[WPR];
      m = q = 0.f;
#pragma unroll
      for (int k = 0; k < WPR; ++k) {
        int c = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int left = D - Part::at(i, 64 * k);
          c += left < 0 ? 0 : left < 64 * VEC ? left : 64 * VEC;
        }
        len[k] = (float)c;
        part[k] = red[turn][0][k];
        m = fmaf(len[k], part[k], m);
      }
      m /= (float)D;
#pragma unroll
      for (int k = 0; k < WPR; ++k) {
        const float d = part[k] - m;
        q += fmaf(len[k] * d, d, red[turn][1][k]);
      }
    }
    const float r = 1.f / sqrtf(q / (float)D + eps);
    if constexpr (kWide) {
      using One = RowPart<T, 1, WPR, WHOLE>;
      const int t0 = opaque(tid);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float g[VEC], b[VEC], *u = v + i * VEC;
        One::columns(gamma, D, t0 + i * WPR * 64, 1.f, g);
        One::columns(beta, D, t0 + i * WPR * 64, 0.f, b);
#pragma unroll
        for (int j = 0; j < VEC; ++j) u[j] = fmaf((u[j] - m) * r, g[j], b[j]);
        One::store(y + here * D, D, t0 + i * WPR * 64, u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = fmaf((v[i] - m) * r, gm[i], bt[i]);
      Part::store(y + here * D, D, tid, v);
    }
    if (tid == 0) {
      if (mean) mean[here] = m;
      if (rstd) rstd[here] = r;
    }
  }
}

// Both sums over the waves of a row, in every lane; `red` is used in turn.
template <int WPR>
__device__ __forceinline__ void block_sums(float& s1, float& s2, float (&red)[2][WPR]) {
  s1 = sum64(s1);
  s2 = sum64(s2);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) {
      red[0][threadIdx.x >> 6] = s1;
      red[1][threadIdx.x >> 6] = s2;
    }
    __syncthreads();
    s1 = s2 = 0.f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) {
      s1 += red[0][i];
      s2 += red[1][i];
    }
  }
}

// Backward over rows.  A block walks over rows as in the forward pass; every lane
// keeps the same columns, so the columns' sums of dgamma and dbeta stay in its
// registers and leave the block once, as row blockIdx of part [2][gridDim][D].
template <typename T, int NV, int WPR, bool WHOLE>
__global__ __launch_bounds__(WPR > 4 ? 64 * WPR : kRowThreads) void norm_rows_bwd_kernel(
    const T* __restrict__ x, const float* __restrict__ gamma, const float* __restrict__ mean,
    const float* __restrict__ rstd, const T* __restrict__ dy, T* __restrict__ dx,
    float* __restrict__ part, long rows, int D) {
  using Part = RowPart<T, NV, WPR, WHOLE>;
  constexpr int VEC = Part::VEC, E = Part::E;
  constexpr int RPB = WPR == 1 ? kRowThreads / 64 : 1;
  __shared__ float red[2][2][WPR];
  __shared__ float cols[WPR == 1 ? 3 * 64 * E : 1];
  const int tid = WPR == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int sub = WPR == 1 ? threadIdx.x >> 6 : 0;
  float gm[E], ag[E], ab[E];
  Part nx, ng;
  float nm = 0.f, nr = 0.f;
  long row = (long)blockIdx.x * RPB + sub;
  if (row < rows) {
    nx.load(x + row * D, D, tid);
    ng.load(dy + row * D, D, tid);
    nm = mean[row];
    nr = rstd[row];
  }
  Part::columns(gamma, D, tid, 1.f, gm);
#pragma unroll
  for (int i = 0; i < E; ++i) ag[i] = ab[i] = 0.f;
  int turn = 0;
  for (; row < rows; turn ^= 1) {
    float xv[E], gv[E];
    nx.get(D, tid, xv);
    ng.get(D, tid, gv);
    const float m = nm, r = nr;
    const long here = row;
    row += (long)gridDim.x * RPB;
    if (row < rows) {
      nx.load(x + row * D, D, tid);
      ng.load(dy + row * D, D, tid);
      nm = mean[row];
      nr = rstd[row];
    }
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      // behind D, dy = 0: nothing is added
      const float xh = (xv[i] - m) * r, w = gv[i] * gm[i];
      xv[i] = xh;
      s1 += w;
      s2 = fmaf(w, xh, s2);
      ag[i] = fmaf(gv[i], xh, ag[i]);
      ab[i] += gv[i];
      gv[i] = w;
    }
    if (dx) {
      block_sums<WPR>(s1, s2, red[turn]);
      s1 /= (float)D;
      s2 /= (float)D;
#pragma unroll
      for (int i = 0; i < E; ++i) gv[i] = r * (gv[i] - s1 - xv[i] * s2);
      Part::store(dx + here * D, D, tid, gv);
    }
  }
  if (!part) return;
  float* pg = part + (size_t)blockIdx.x * D;
  float* pb = part + ((size_t)gridDim.x + blockIdx.x) * D;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float* a = half ? ab : ag;
    if constexpr (WPR == 1) {
      // the four waves hold the same columns
      __syncthreads();
      if (sub)
#pragma unroll
        for (int i = 0; i < E; ++i) cols[((sub - 1) * E + i) * 64 + tid] = a[i];
      __syncthreads();
      if (sub) continue;
#pragma unroll
      for (int i = 0; i < E; ++i)
        a[i] += (cols[i * 64 + tid] + cols[(E + i) * 64 + tid]) + cols[(2 * E + i) * 64 + tid];
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = Part::at(i, tid);
      float* o = (half ? pb : pg) + c;
      if (c + VEC <= D) {
        __builtin_memcpy(o, a + i * VEC, VEC * sizeof(float));
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (c + j < D) o[j] = a[i * VEC + j];
      }
    }
  }
}

// Backward over wide rows, in two kernels, since a row's columns leave no registers for
// their sums: dx by rows (x and dy are read again behind the row's sums, from the
// caches), and the columns' sums.
template <typename T, int WPR, bool WHOLE>
__global__ __launch_bounds__(64 * WPR) void norm_wide_dx_kernel(
    const T* __restrict__ x, const float* __restrict__ gamma, const float* __restrict__ mean,
    const float* __restrict__ rstd, const T* __restrict__ dy, T* __restrict__ dx, long rows,
    int D) {
  using One = RowPart<T, 1, WPR, WHOLE>;
  constexpr int VEC = One::VEC, STEP = 64 * WPR;
  __shared__ float red[2][2][WPR];
  const int tid = threadIdx.x;
  int turn = 0;
  for (long row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
    const T *xr = x + row * D, *gr = dy + row * D;
    T* dr = dx + row * D;
    const float m = mean[row], r = rstd[row];
    auto vectors = [&](auto f) {   // f(at, xh, dy gamma); a whole step is inside or partly
      One xo, go;
      float xv[VEC], gv[VEC], g[VEC];
#pragma unroll 2
      for (int at = tid; at * VEC < D; at += STEP) {
        xo.load(xr, D, at);
        go.load(gr, D, at);
        One::columns(gamma, D, at, 1.f, g);
        xo.get(D, at, xv);
        go.get(D, at, gv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          xv[j] = (xv[j] - m) * r;
          gv[j] *= g[j];
        }
        f(at, xv, gv);
      }
    };
    float s1 = 0.f, s2 = 0.f;
    vectors([&](int, const float* xh, const float* w) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {   // behind D, w = 0: nothing is added
        s1 += w[j];
        s2 = fmaf(w[j], xh[j], s2);
      }
    });
    block_sums<WPR>(s1, s2, red[turn]);
    s1 /= (float)D;
    s2 /= (float)D;
    vectors([&](int at, const float* xh, const float* w) {
      float o[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = r * (w[j] - s1 - xh[j] * s2);
      One::store(dr, D, at, o);
    });
  }
}

// Block: 64 vectors of columns, the rows blockIdx.y 4 + wave and on by gridDim.y 4.
template <typename T, bool WHOLE>
__global__ __launch_bounds__(256) void norm_wide_sums_kernel(
    const T* __restrict__ x, const float* __restrict__ mean, const float* __restrict__ rstd,
    const T* __restrict__ dy, float* __restrict__ part, long rows, int D) {
  using One = RowPart<T, 1, 1, WHOLE>;
  constexpr int VEC = One::VEC;
  __shared__ float red[3][2][VEC][64];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int at = blockIdx.x * 64 + lane;
  float ag[VEC], ab[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) ag[j] = ab[j] = 0.f;
#pragma unroll 4
  for (long row = blockIdx.y * 4 + w; row < rows; row += gridDim.y * 4) {
    One xo, go;
    float xv[VEC], gv[VEC];
    xo.load(x + row * D, D, at);
    go.load(dy + row * D, D, at);
    const float m = mean[row], r = rstd[row];
    xo.get(D, at, xv);
    go.get(D, at, gv);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      ag[j] = fmaf(gv[j], (xv[j] - m) * r, ag[j]);
      ab[j] += gv[j];
    }
  }
  if (w > 0)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      red[w - 1][0][j][lane] = ag[j];
      red[w - 1][1][j][lane] = ab[j];
    }
  __syncthreads();
  if (w > 0) return;
  float* pg = part + (size_t)blockIdx.y * D;
  float* pb = part + ((size_t)gridDim.y + blockIdx.y) * D;
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const int c = at * VEC + j;
    if (c >= D) continue;
    pg[c] = ag[j] + ((red[0][0][j][lane] + red[1][0][j][lane]) + red[2][0][j][lane]);
    pb[c] = ab[j] + ((red[0][1][j][lane] + red[1][1][j][lane]) + red[2][1][j][lane]);
  }
}

// dgamma[c] = sum_b part[0][b][c], dbeta[c] = sum_b part[1][b][c], always in the
// same order.  Block: 32 columns (a line); 32 groups of lanes share the partial rows.
__global__ __launch_bounds__(1024) void norm_columns_kernel(const float* __restrict__ part, int nb,
                                                            int D, float* __restrict__ dgamma,
                                                            float* __restrict__ dbeta) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float* out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  const float* p = part + (size_t)blockIdx.y * nb * D;
  float s = 0.f;
  if (c < D)
#pragma unroll 8
    for (int b = w; b < nb; b += 32) s += p[(size_t)b * D + c];
  red[w][lane] = s;
  __syncthreads();
  // group w adds up column w
  float t = red[lane][w];
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) t += __shfl_xor(t, off);
  const int col = blockIdx.x * 32 + w;
  if (lane == 0 && col < D) out[col] = t;
}

// ------------------------------------------------------- inner > 1: channels

// Lanes take 64 neighbouring positions (o, i) of the flattened outer x inner
// axis, so a wave reads a line of one channel; the block's 8 waves take the
// channels d = w, w + 8, ...  EPT > 0 (D <= 8 EPT): the values stay in
// registers; EPT = 0: they are read again, from the caches where they fit.
constexpr int kChWaves = 8;

template <int NS>
__device__ __forceinline__ void wave_sums(float (&s)[NS], float (*red)[kChWaves][64], int w,
                                          int lane) {
#pragma unroll
  for (int k = 0; k < NS; ++k) red[k][w][lane] = s[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kChWaves; ++i) t += red[k][i][lane];
    s[k] = t;
  }
}

template <typename T, int EPT>
__global__ __launch_bounds__(64 * kChWaves) void norm_channels_kernel(
    const T* x, const float* __restrict__ gamma, const float* __restrict__ beta, T* y,
    float* __restrict__ mean, float* __restrict__ rstd, long outer, int D, long inner, float eps) {
  __shared__ float red[2][1][kChWaves][64];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const long pos = (long)blockIdx.x * 64 + lane;
  const bool on = pos < outer * inner;
  const long o = on ? pos / inner : 0, i0 = on ? pos - o * inner : 0;
  const T* xp = x + o * D * inner + i0;
  float v[EPT > 0 ? EPT : 1];
  float s[1] = {0.f};
  if constexpr (EPT > 0) {
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
      const int d = w + kChWaves * k;
      v[k] = on && d < D ? to_f32(xp[d * inner]) : 0.f;
      s[0] += v[k];
    }
  } else if (on) {
#pragma unroll 8
    for (int d = w; d < D; d += kChWaves) s[0] += to_f32(xp[d * inner]);
  }
  wave_sums(s, red[0], w, lane);
  const float m = s[0] / (float)D;
  s[0] = 0.f;
  if constexpr (EPT > 0) {
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
      v[k] -= m;
      s[0] += w + kChWaves * k < D ? v[k] * v[k] : 0.f;
    }
  } else if (on) {
#pragma unroll 8
    for (int d = w; d < D; d += kChWaves) {
      const float t = to_f32(xp[d * inner]) - m;
      s[0] = fmaf(t, t, s[0]);
    }
  }
  wave_sums(s, red[1], w, lane);
  const float r = 1.f / sqrtf(s[0] / (float)D + eps);
  if (!on) return;
  T* yp = y + o * D * inner + i0;
  if constexpr (EPT > 0) {
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
      const int d = w + kChWaves * k;
      if (d < D)
        yp[d * inner] = from_f32<T>(
            fmaf(v[k] * r, gamma ? gamma[d] : 1.f, beta ? beta[d] : 0.f));
    }
  } else {
#pragma unroll 8
    for (int d = w; d < D; d += kChWaves)
      yp[d * inner] = from_f32<T>(fmaf((to_f32(xp[d * inner]) - m) * r, gamma ? gamma[d] : 1.f,
                                       beta ? beta[d] : 0.f));
  }
  if (w == 0) {
    if (mean) mean[pos] = m;
    if (rstd) rstd[pos] = r;
  }
}

// Backward: a block walks over tiles of 64 positions.  EPT > 0: dgamma and dbeta
// of the thread's channels are summed in registers over the tiles and over the
// lanes at the end; EPT = 0: over the lanes in every tile, into the block's own
// row of part (no other block touches it).
template <typename T, int EPT>
__global__ __launch_bounds__(64 * kChWaves) void norm_channels_bwd_kernel(
    const T* __restrict__ x, const float* __restrict__ gamma, const float* __restrict__ mean,
    const float* __restrict__ rstd, const T* __restrict__ dy, T* __restrict__ dx,
    float* __restrict__ part, long outer, int D, long inner) {
  __shared__ float red[2][2][kChWaves][64];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const long positions = outer * inner, tiles = (positions + 63) / 64;
  float* pg = part ? part + (size_t)blockIdx.x * D : nullptr;
  float* pb = part ? part + ((size_t)gridDim.x + blockIdx.x) * D : nullptr;
  constexpr int E = EPT > 0 ? EPT : 1;
  float ag[E], ab[E];
#pragma unroll
  for (int k = 0; k < E; ++k) ag[k] = ab[k] = 0.f;
  int turn = 0;
  bool first = true;
  for (long tile = blockIdx.x; tile < tiles; tile += gridDim.x, turn ^= 1, first = false) {
    const long pos = tile * 64 + lane;
    const bool on = pos < positions;
    const long o = on ? pos / inner : 0, i0 = on ? pos - o * inner : 0;
    const T* xp = x + o * D * inner + i0;
    const T* gp = dy + o * D * inner + i0;
    T* dp = dx ? dx + o * D * inner + i0 : nullptr;
    const float m = on ? mean[pos] : 0.f, r = on ? rstd[pos] : 0.f;
    float s[2] = {0.f, 0.f};
    float xh[E], wv[E];
    if constexpr (EPT > 0) {
#pragma unroll
      for (int k = 0; k < EPT; ++k) {
        const int d = w + kChWaves * k;
        const bool in = on && d < D;
        xh[k] = in ? to_f32(xp[d * inner]) : 0.f;
        wv[k] = in ? to_f32(gp[d * inner]) : 0.f;
      }
#pragma unroll
      for (int k = 0; k < EPT; ++k) {
        const int d = w + kChWaves * k;
        const float g = wv[k];
        xh[k] = (xh[k] - m) * r;
        ag[k] = fmaf(g, xh[k], ag[k]);
        ab[k] += g;
        wv[k] = g * (gamma && d < D ? gamma[d] : 1.f);
        s[0] += wv[k];
        s[1] = fmaf(wv[k], xh[k], s[1]);
      }
    } else {
      for (int d = w; d < D; d += kChWaves) {
        const float g = on ? to_f32(gp[d * inner]) : 0.f;
        const float h = on ? (to_f32(xp[d * inner]) - m) * r : 0.f;
        const float wg = g * (gamma ? gamma[d] : 1.f);
        s[0] += wg;
        s[1] = fmaf(wg, h, s[1]);
        if (part) {
          const float tg = sum64(g * h), tb = sum64(g);
          if (lane == 0) {
            pg[d] = first ? tg : pg[d] + tg;
            pb[d] = first ? tb : pb[d] + tb;
          }
        }
      }
    }
    if (!dx) continue;
    wave_sums(s, red[turn], w, lane);
    const float a = s[0] / (float)D, b = s[1] / (float)D;
    if (!on) continue;   // no barrier behind this
    if constexpr (EPT > 0) {
#pragma unroll
      for (int k = 0; k < EPT; ++k) {
        const int d = w + kChWaves * k;
        if (d < D) dp[d * inner] = from_f32<T>(r * (wv[k] - a - xh[k] * b));
      }
    } else {
#pragma unroll 4
      for (int d = w; d < D; d += kChWaves) {
        const float h = (to_f32(xp[d * inner]) - m) * r;
        const float wg = to_f32(gp[d * inner]) * (gamma ? gamma[d] : 1.f);
        dp[d * inner] = from_f32<T>(r * (wg - a - h * b));
      }
    }
  }
  if constexpr (EPT == 0) {
    if (part && first)   // no positions at all
      for (int d = threadIdx.x; d < D; d += 64 * kChWaves) pg[d] = pb[d] = 0.f;
  } else {
    if (!part) return;
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
      const int d = w + kChWaves * k;
      const float tg = sum64(ag[k]), tb = sum64(ab[k]);
      if (lane == 0 && d < D) {
        pg[d] = tg;
        pb[d] = tb;
      }
    }
  }
}

long ceil_div(long a, long b) { return (a + b - 1) / b; }

// Vectors a lane holds and waves a row takes: one wave up to 2 vectors a lane, then
// 4 waves, then 16.
template <typename T, typename F>
void row_shape(int D, F f) {
  const int vecs = (int)ceil_div(D, 64 * Vec<T>::N);
  const bool whole = D % Vec<T>::N == 0;
  using std::integral_constant;
  using Yes = std::true_type;
  using No = std::false_type;
#define S4_CASE(nv, wpr)                                                                 \
  (whole ? f(integral_constant<int, nv>(), integral_constant<int, wpr>(), Yes())         \
         : f(integral_constant<int, nv>(), integral_constant<int, wpr>(), No()))
  if (vecs <= 1) return S4_CASE(1, 1);
  if (vecs <= 2) return S4_CASE(2, 1);
  if (vecs <= 4) return S4_CASE(1, 4);
  if (vecs <= 8) return S4_CASE(2, 4);
  if (vecs <= 16) return S4_CASE(4, 4);
  if (vecs <= 32) return S4_CASE(2, 16);
  if (vecs <= 64) return S4_CASE(4, 16);
  if constexpr (sizeof(T) == 4) return S4_CASE(8, 16);
#undef S4_CASE
}

template <typename T>
hipError_t fwd(const NormArgs& a, hipStream_t s) {
  const T* x = (const T*)a.x;
  T* y = (T*)a.y;
  const int D = (int)a.D;
  if (a.inner == 1) {
    row_shape<T>(D, [&](auto nv, auto wpr, auto whole) {
      constexpr int NV = decltype(nv)::value, WPR = decltype(wpr)::value;
      constexpr bool W = decltype(whole)::value;
      const long blocks = WPR == 1 ? ceil_div(a.outer, kRowThreads / 64) : a.outer;
      const long most = WPR > 4 ? kNormBlocks / 4 : kNormBlocks;
      norm_rows_kernel<T, NV, WPR, W>
          <<<dim3((unsigned)(blocks < most ? blocks : most)), WPR > 4 ? 64 * WPR : kRowThreads, 0,
             s>>>(x, a.gamma, a.beta, y, a.mean, a.rstd, a.outer, D, a.eps);
    });
    return hipGetLastError();
  }
  const dim3 grid((unsigned)ceil_div(a.outer * a.inner, 64));
#define S4_GO(ept)                                                                            \
  norm_channels_kernel<T, ept><<<grid, 64 * kChWaves, 0, s>>>(x, a.gamma, a.beta, y, a.mean,  \
                                                              a.rstd, a.outer, D, a.inner, a.eps)
  if (D <= 8 * kChWaves) S4_GO(8);
  else if (D <= 32 * kChWaves) S4_GO(32);
  else if (D <= 64 * kChWaves) S4_GO(64);
  else S4_GO(0);
#undef S4_GO
  return hipGetLastError();
}

template <typename T>
hipError_t bwd(const NormArgs& a, hipStream_t s) {
  const T *x = (const T*)a.x, *dy = (const T*)a.dy;
  T* dx = (T*)a.dx;
  const int D = (int)a.D;
  const bool sums = a.dgamma || a.dbeta;
  float* part = sums ? a.part : nullptr;
  const int nb = (int)norm_parts(a.outer, a.D, a.inner);
  if (a.inner == 1) {
    row_shape<T>(D, [&](auto nv, auto wpr, auto whole) {
      constexpr int NV = decltype(nv)::value, WPR = decltype(wpr)::value;
      constexpr bool W = decltype(whole)::value;
      if constexpr (wide_rows(NV * Vec<T>::N, WPR)) {
        if (dx && a.outer > 0)
          norm_wide_dx_kernel<T, WPR, W>
              <<<dim3((unsigned)(a.outer < 512 ? a.outer : 512)), 64 * WPR, 0, s>>>(
                  x, a.gamma, a.mean, a.rstd, dy, dx, a.outer, D);
        if (part)
          norm_wide_sums_kernel<T, W>
              <<<dim3((unsigned)ceil_div(D, 64 * Vec<T>::N), nb), 256, 0, s>>>(
                  x, a.mean, a.rstd, dy, part, a.outer, D);
      } else {
        norm_rows_bwd_kernel<T, NV, WPR, W>
            <<<dim3(nb), WPR > 4 ? 64 * WPR : kRowThreads, 0, s>>>(x, a.gamma, a.mean, a.rstd, dy,
                                                                   dx, part, a.outer, D);
      }
    });
  } else {
#define S4_GO(ept)                                                                   \
  norm_channels_bwd_kernel<T, ept><<<dim3(nb), 64 * kChWaves, 0, s>>>(               \
      x, a.gamma, a.mean, a.rstd, dy, dx, part, a.outer, D, a.inner)
    if (D <= 8 * kChWaves) S4_GO(8);
    else if (D <= 32 * kChWaves) S4_GO(32);
    else S4_GO(0);
#undef S4_GO
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !sums) return e;
  norm_columns_kernel<<<dim3((unsigned)ceil_div(D, 32), 2), 1024, 0, s>>>(part, nb, D, a.dgamma,
                                                                         a.dbeta);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs& a, int dtype, hipStream_t s) {
  return dtype == S4DPLR_F32 ? fwd<float>(a, s) : dtype == S4DPLR_BF16 ? fwd<bf16>(a, s) : fwd<f16>(a, s);
}

hipError_t launch_norm_bwd(const NormArgs& a, int dtype, hipStream_t s) {
  return dtype == S4DPLR_F32 ? bwd<float>(a, s) : dtype == S4DPLR_BF16 ? bwd<bf16>(a, s) : bwd<f16>(a, s);
}

}  // namespace s4
