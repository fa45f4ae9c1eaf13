// Layer norm, forward and backward, over the middle axis of x [outer][D][inner]:
//   m = mean_d x,  r = 1 / sqrt(mean_d (x - m)^2 + eps),  y = (x - m) r gamma + beta,
//   xh = (x - m) r,  w = dy gamma,
//   dx = r (w - mean_d w - xh mean_d (w xh)),  dgamma = sum dy xh,  dbeta = sum dy.
// inner = 1 is the token-major layout (rows of D contiguous values), inner = L
// the [batch][H][L] layout normalized over its H channels.  Elements are fp32,
// bf16 or fp16; all arithmetic is fp32, each output is rounded once.  The
// variance is the mean of squared deviations from the mean (two passes over
// registers).  A mean m of fp32 sums is off by some of its own steps c, which counts
// where values are large against their spread; the second pass finds it,
//   c = sum (x - m) / D,  mean = m + c,  variance = sum (x - m)^2 / D - c^2,
// which is applied where c is more than 2^-20 of the deviation (below, the sum's own rounding
// is no smaller).
//
// Both directions are bound by HBM: forward reads x and writes y, backward reads
// x and dy and writes dx.  Measured, bf16 rows: forward of 16384 x 4096 47 us (5.7 TB/s,
// part of it from the last-level cache), backward of 16384 x 2048 42 us with the columns'
// sums (4.8 TB/s); fp32 channels 32 x 256 x 1024: 15.5 us (4.3 TB/s) and 25.4 us (4.0
// TB/s); bf16 channels 11.8 us (2.8 TB/s) and 19.9 us (2.5 TB/s).
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

// Rows of 32 values a lane over 16 waves: those have 128 registers a lane, so gamma and beta
// are read where they are used (2048 x 32768 bf16 108 -> 72 us; 60 since the forward pass joins
// its waves' parts a lane each, which leaves it without spills; fp32 114).
constexpr bool wide_rows(int values, int waves) { return waves > 4 && values > 16; }

// The same value, unknown to the compiler: a load at it is not taken out of the loop, where
// its result would be kept in registers and spilled.
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Sum over every group of N lanes, 4 or 16, the same bits in all of them: a lane's own product
// must not enter the first addition unrounded, as a contraction would have it.
template <int N>
__device__ __forceinline__ float sum_of(float v) {
#pragma clang fp contract(off)
  static_assert(N == 4 || N == 16, "");
  v += dpp<0xB1>(v);    // quad_perm [1, 0, 3, 2]
  v += dpp<0x4E>(v);    // quad_perm [2, 3, 0, 1]
  if constexpr (N == 16) {
    v += dpp<0x141>(v);   // row_half_mirror
    v += dpp<0x140>(v);   // row_mirror
  }
  return v;
}

// The error that counts of a mean of n values, from the sums e of what they differ by and q
// of its squares; 0 too where either is not finite.
__device__ __forceinline__ float lost(float e, float q, float n) {
  const float c = e / n;
  return c * e > 0x1p-40f * q ? c : 0.f;
}

// Forward over rows.  WPR waves share a row (blocks of 256 threads hold 4 rows at WPR =
// 1), and a block walks over rows blockIdx, blockIdx + gridDim, ..., the next row on its
// way while one is computed: gamma and beta are read once.  A wave takes mean (m_w + c_w)
// and squared deviations M_w of its own part; the parts are joined by
//   m = sum n_w m_w / D,  t_w = (m_w - m) + c_w,  c = sum n_w t_w / D,  mean = m + c,
//   M = sum (M_w + n_w t_w^2) - D c^2,
// with one barrier a row (two sets of slots in turn).
template <typename T, int NV, int WPR, bool WHOLE>
__global__ __launch_bounds__(WPR > 4 ? 64 * WPR : kRowThreads) void norm_rows_kernel(
    const T* x, const float* __restrict__ gamma, const float* __restrict__ beta, T* y,
    float* __restrict__ mean, float* __restrict__ rstd, long rows, int D, float eps) {
  using Part = RowPart<T, NV, WPR, WHOLE>;
  constexpr int VEC = Part::VEC, E = Part::E;
  constexpr int RPB = WPR == 1 ? kRowThreads / 64 : 1;
  __shared__ float red[2][3][WPR];
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
  // elements of the wave's part, and of part lane % WPR
  float n = (float)D, n_of = n;
  if constexpr (WPR > 1) {
    auto elements = [&](int k) {
      int c = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int left = D - Part::at(i, 64 * k);
        c += left < 0 ? 0 : left < 64 * VEC ? left : 64 * VEC;
      }
      return (float)c;
    };
    n = elements(w);
    n_of = elements(tid % WPR);
  }
  int turn = 0;
  for (; row < rows; turn ^= 1) {
    float v[E];
    next.get(D, tid, v);
    const long here = row;
    row += (long)gridDim.x * RPB;
    if (row < rows) next.load(x + row * D, D, tid);
    float s = 0.f, q = 0.f, e = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s += v[i];
    float m = n > 0.f ? sum64(s) / n : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float d = Part::at(i, tid) + j < D ? v[i * VEC + j] - m : 0.f;
        q = fmaf(d, d, q);
        e += d;
      }
    e = sum64(e);
    q = sum64(q);
    float c = lost(e, q, n);
    q -= e * c;
    if constexpr (WPR == 1) {
      m += c;
    } else {
      if (tid % 64 == 0) {
        red[turn][0][w] = m;
        red[turn][1][w] = q;
        red[turn][2][w] = c;
      }
      __syncthreads();
      // every lane one part, and sums over the WPR lanes
      const int k = tid % WPR;
      m = sum_of<WPR>(n_of * red[turn][0][k]) / (float)D;
      const float part = (red[turn][0][k] - m) + red[turn][2][k];
      e = sum_of<WPR>(n_of * part);
      q = sum_of<WPR>(fmaf(n_of * part, part, red[turn][1][k]));
      c = lost(e, q, (float)D);
      q -= e * c;
      m += c;
    }
    q = q < 0.f ? 0.f : q;   // NaN stays
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
// registers and leave the block once, as row blockIdx of part [2][gridDim][D].  Rows of 8193 to
// 16384 values spill (fp32 44 registers a lane; 16 bits 17, and 72 where D is no multiple of 8):
// 4096 x 16384 117 us in bf16 and 248 in fp32, 1.5 times what a copy of their bytes takes,
// 4096 x 16380 bf16 176.
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
// caches), and the columns' sums.  2048 x 32768 bf16 156 us (in one kernel, which spilled,
// 639), 512 x 32768 fp32 76 (314).
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

// Lanes take neighbouring positions (o, i) of the flattened outer x inner axis, so a wave
// reads a line of one channel; the block's W waves take the channels d = w, w + W, ....
// VP positions a lane: two of 16 bits where inner is even, so that they lie side by
// side.  EPT > 0 (D <= W EPT): a lane's elements stay in its registers as they came;
// EPT = 0: they are read again, from the caches where they fit.
template <typename T, int VP>
struct Pack {
  T v[VP];
};
template <typename T, int VP>
__device__ __forceinline__ Pack<T, VP> load_pack(const T* p) {
  Pack<T, VP> r;
  __builtin_memcpy(&r, p, sizeof(r));
  return r;
}
// Channel d of D at a lane's positions.  Elements of 16 bits are read without a branch, a
// missing one from channel 0 (a load into half a register is waited for at a branch: 59
// us instead of 30 for the gradients of 32 x 256 x 1024 bf16, with 8 waves); of 32 bits,
// under the condition (33.0 us against 35.4 in fp32).  What a missing one holds is not used.
template <typename T, int VP>
__device__ __forceinline__ Pack<T, VP> load_channel(const T* p, int d, int D, unsigned inner,
                                                    bool on) {
  if constexpr (sizeof(T) == 2) return load_pack<T, VP>(p + (long)(d < D ? d : 0) * inner);
  Pack<T, VP> r = {};
  if (on && d < D) r = load_pack<T, VP>(p + (long)d * inner);
  return r;
}
// Two floats of a converted pair are not worth keeping for the next pass.
template <typename T, int VP>
__device__ __forceinline__ void forget(Pack<T, VP>& x) {
  if constexpr (sizeof(x) == 4) {
    int t;
    __builtin_memcpy(&t, &x, 4);
    t = opaque(t);
    __builtin_memcpy(&x, &t, 4);
  }
}

// s[k] summed over the block's waves, position by position.
template <int NS, int W, int VP>
__device__ __forceinline__ void wave_sums(float (&s)[NS][VP], float (*red)[W][64 * VP], int w,
                                          int lane) {
#pragma unroll
  for (int k = 0; k < NS; ++k)
#pragma unroll
    for (int q = 0; q < VP; ++q) red[k][w][lane * VP + q] = s[k][q];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < NS; ++k)
#pragma unroll
    for (int q = 0; q < VP; ++q) {
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) t += red[k][i][lane * VP + q];
      s[k][q] = t;
    }
}

// Where a lane's positions lie.
template <int VP>
struct Positions {
  bool on;
  unsigned pos;
  long at;   // element of channel 0
  __device__ __forceinline__ Positions(unsigned tile, int lane, unsigned positions, int D,
                                       unsigned inner) {
    pos = (tile * 64 + lane) * VP;
    on = pos < positions;
    const unsigned o = on ? pos / inner : 0;
    at = (long)o * D * inner + (on ? pos - o * inner : 0);
  }
};

template <typename T, int EPT, int W, int VP>
__global__ __launch_bounds__(64 * W) void norm_channels_kernel(
    const T* x, const float* __restrict__ gamma, const float* __restrict__ beta, T* y,
    float* __restrict__ mean, float* __restrict__ rstd, unsigned positions, int D, unsigned inner,
    float eps) {
  using P = Pack<T, VP>;
  __shared__ float red0[1][W][64 * VP], red1[2][W][64 * VP];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned tiles = (positions + 64 * VP - 1) / (64 * VP);
  for (unsigned tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const Positions<VP> ps(tile, lane, positions, D, inner);
    const bool on = ps.on;
    const T* xp = x + ps.at;
    P v[EPT > 0 ? EPT : 1];
    // every channel of the wave: f(k, d)
    auto channels = [&](auto f) {
      if constexpr (EPT > 0) {
#pragma unroll
        for (int k = 0; k < EPT; ++k) f(k, w + W * k);
      } else {
#pragma unroll 8
        for (int d = w; d < D; d += W) {
          v[0] = load_channel<T, VP>(xp, d, D, inner, on);
          f(0, d);
        }
      }
    };
    if constexpr (EPT > 0)
#pragma unroll
      for (int k = 0; k < EPT; ++k) v[k] = load_channel<T, VP>(xp, w + W * k, D, inner, on);
    // Many channels: a wave sums differences from its first one, since thousands of additions
    // after one another would leave the mean more than a few steps off.
    float s[1][VP], e[2][VP], x0[VP], m[VP], r[VP];
#pragma unroll
    for (int q = 0; q < VP; ++q) s[0][q] = e[0][q] = e[1][q] = x0[q] = 0.f;
    if constexpr (EPT == 0) {
      const P t = load_channel<T, VP>(xp, w, D, inner, on);
#pragma unroll
      for (int q = 0; q < VP; ++q) x0[q] = w < D ? to_f32(t.v[q]) : 0.f;
    }
    channels([&](int k, int d) {
#pragma unroll
      for (int q = 0; q < VP; ++q) s[0][q] += d < D ? to_f32(v[k].v[q]) - x0[q] : 0.f;
      if constexpr (EPT > 0) forget(v[k]);
    });
    if constexpr (EPT == 0)
#pragma unroll
      for (int q = 0; q < VP; ++q) s[0][q] = fmaf((float)((D - w + W - 1) / W), x0[q], s[0][q]);
    wave_sums<1, W, VP>(s, red0, w, lane);
#pragma unroll
    for (int q = 0; q < VP; ++q) m[q] = s[0][q] / (float)D;
    channels([&](int k, int d) {
#pragma unroll
      for (int q = 0; q < VP; ++q) {
        const float t = d < D ? to_f32(v[k].v[q]) - m[q] : 0.f;
        e[0][q] = fmaf(t, t, e[0][q]);
        e[1][q] += t;
      }
      if constexpr (EPT > 0) forget(v[k]);
    });
    wave_sums<2, W, VP>(e, red1, w, lane);
#pragma unroll
    for (int q = 0; q < VP; ++q) {
      const float c = lost(e[1][q], e[0][q], (float)D), sq = e[0][q] - e[1][q] * c;
      m[q] += c;
      r[q] = 1.f / sqrtf((sq < 0.f ? 0.f : sq) / (float)D + eps);   // NaN stays
    }
    if (!on) continue;   // red0 is free: every wave has passed the second barrier
    T* yp = y + ps.at;
    channels([&](int k, int d) {
      if (d >= D) return;
      const float g = gamma ? gamma[d] : 1.f, b = beta ? beta[d] : 0.f;
      P t;
#pragma unroll
      for (int q = 0; q < VP; ++q)
        t.v[q] = from_f32<T>(fmaf((to_f32(v[k].v[q]) - m[q]) * r[q], g, b));
      __builtin_memcpy(yp + (long)d * inner, &t, sizeof(t));
    });
    if (w == 0)
#pragma unroll
      for (int q = 0; q < VP; ++q) {
        if (mean) mean[ps.pos + q] = m[q];
        if (rstd) rstd[ps.pos + q] = r[q];
      }
  }
}

// dx alone, for more channels than the fused kernel holds sums of (32 x 256 x 1024: fused
// 25.9 us in fp32 and 20.2 in bf16, apart 45.4 and 24.5).  x and dy are read again for dx,
// from the caches (kept in registers, up to 512 channels: 58.3 us instead of 40.5 with the
// sums for 32 x 512 x 1024 bf16, 77.5 instead of 72.7 in fp32).
template <typename T, int W, int VP>
__global__ __launch_bounds__(64 * W) void norm_channels_dx_kernel(
    const T* __restrict__ x, const float* __restrict__ gamma, const float* __restrict__ mean,
    const float* __restrict__ rstd, const T* __restrict__ dy, T* __restrict__ dx,
    unsigned positions, int D, unsigned inner) {
  using P = Pack<T, VP>;
  __shared__ float red[2][2][W][64 * VP];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned tiles = (positions + 64 * VP - 1) / (64 * VP);
  int turn = 0;
  for (unsigned tile = blockIdx.x; tile < tiles; tile += gridDim.x, turn ^= 1) {
    const Positions<VP> ps(tile, lane, positions, D, inner);
    const bool on = ps.on;
    float m[VP], r[VP];
#pragma unroll
    for (int q = 0; q < VP; ++q) {
      m[q] = on ? mean[ps.pos + q] : 0.f;
      r[q] = on ? rstd[ps.pos + q] : 0.f;
    }
    auto channels = [&](auto f) {   // f(d, xh, dy gamma)
#pragma unroll 4
      for (int d = w; d < D; d += W) {
        const P v = load_channel<T, VP>(x + ps.at, d, D, inner, on);
        const P g = load_channel<T, VP>(dy + ps.at, d, D, inner, on);
        const float gm = gamma ? gamma[d] : 1.f;
        float xh[VP], wg[VP];
#pragma unroll
        for (int q = 0; q < VP; ++q) {
          xh[q] = (to_f32(v.v[q]) - m[q]) * r[q];
          wg[q] = to_f32(g.v[q]) * gm;
        }
        f(d, xh, wg);
      }
    };
    float s[2][VP];
#pragma unroll
    for (int q = 0; q < VP; ++q) s[0][q] = s[1][q] = 0.f;
    channels([&](int, const float* xh, const float* wg) {
#pragma unroll
      for (int q = 0; q < VP; ++q) {
        s[0][q] += wg[q];
        s[1][q] = fmaf(wg[q], xh[q], s[1][q]);
      }
    });
    wave_sums<2, W, VP>(s, red[turn], w, lane);
#pragma unroll
    for (int q = 0; q < VP; ++q) {
      s[0][q] /= (float)D;
      s[1][q] /= (float)D;
    }
    if (!on) continue;   // no barrier behind this
    channels([&](int d, const float* xh, const float* wg) {
      P t;
#pragma unroll
      for (int q = 0; q < VP; ++q) t.v[q] = from_f32<T>(r[q] * (wg[q] - s[0][q] - xh[q] * s[1][q]));
      __builtin_memcpy(dx + ps.at + (long)d * inner, &t, sizeof(t));
    });
  }
}

// The columns' sums for the same: a wave takes kSums channels, its lanes V positions
// each (16 bytes where inner is a multiple of them, else one), and the block's row of
// part the tiles blockIdx.y, blockIdx.y + gridDim.y, ....
constexpr int kSums = 4;

template <typename T, int V>
__global__ __launch_bounds__(256) void norm_channels_sums_kernel(
    const T* __restrict__ x, const float* __restrict__ mean, const float* __restrict__ rstd,
    const T* __restrict__ dy, float* __restrict__ part, unsigned positions, int D,
    unsigned inner) {
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int d0 = (blockIdx.x * 4 + w) * kSums;
  if (d0 >= D) return;
  const unsigned tiles = (positions + 64 * V - 1) / (64 * V);
  float ag[kSums], ab[kSums];
#pragma unroll
  for (int c = 0; c < kSums; ++c) ag[c] = ab[c] = 0.f;
  for (unsigned tile = blockIdx.y; tile < tiles; tile += gridDim.y) {
    const Positions<V> ps(tile, lane, positions, D, inner);
    if (!ps.on) continue;
    float m[V], r[V];
    __builtin_memcpy(m, mean + ps.pos, sizeof(m));
    __builtin_memcpy(r, rstd + ps.pos, sizeof(r));
    Pack<T, V> v[kSums], g[kSums];
#pragma unroll
    for (int c = 0; c < kSums; ++c) {   // channels behind D: the last one, not written
      const long at = ps.at + (long)(d0 + c < D ? d0 + c : D - 1) * inner;
      v[c] = load_pack<T, V>(x + at);
      g[c] = load_pack<T, V>(dy + at);
    }
#pragma unroll
    for (int c = 0; c < kSums; ++c)
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const float t = to_f32(g[c].v[q]);
        ag[c] = fmaf(t, (to_f32(v[c].v[q]) - m[q]) * r[q], ag[c]);
        ab[c] += t;
      }
  }
#pragma unroll
  for (int c = 0; c < kSums; ++c) {
    const float tg = sum64(ag[c]), tb = sum64(ab[c]);
    if (lane == 0 && d0 + c < D) {
      part[(size_t)blockIdx.y * D + d0 + c] = tg;
      part[((size_t)gridDim.y + blockIdx.y) * D + d0 + c] = tb;
    }
  }
}

// Backward, up to W EPT channels: a block walks over tiles of 64 positions; dgamma and
// dbeta of the thread's channels are summed in registers over the tiles and over the
// lanes at the end.  Above 64 channels 16 waves of 16 channels at one block a CU (32 x 256 x
// 1024 fp32 25.9 us; 8 waves of 32 channels, two blocks a CU launched, took 34.6).
template <typename T, int EPT, int W>
__global__ __launch_bounds__(64 * W) void norm_channels_bwd_kernel(
    const T* __restrict__ x, const float* __restrict__ gamma, const float* __restrict__ mean,
    const float* __restrict__ rstd, const T* __restrict__ dy, T* __restrict__ dx,
    float* __restrict__ part, unsigned positions, int D, unsigned inner) {
  __shared__ float red[2][2][W][64];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned tiles = (positions + 63) / 64;
  float ag[EPT], ab[EPT];
#pragma unroll
  for (int k = 0; k < EPT; ++k) ag[k] = ab[k] = 0.f;
  int turn = 0;
  for (unsigned tile = blockIdx.x; tile < tiles; tile += gridDim.x, turn ^= 1) {
    const Positions<1> ps(tile, lane, positions, D, inner);
    const bool on = ps.on;
    const T *xp = x + ps.at, *gp = dy + ps.at;
    const float m = on ? mean[ps.pos] : 0.f, r = on ? rstd[ps.pos] : 0.f;
    float s[2][1] = {{0.f}, {0.f}};
    float xh[EPT], wv[EPT];
    Pack<T, 1> xr[EPT], gr[EPT];
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
      xr[k] = load_channel<T, 1>(xp, w + W * k, D, inner, on);
      gr[k] = load_channel<T, 1>(gp, w + W * k, D, inner, on);
    }
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
      const int d = w + W * k;
      const bool in = on && d < D;
      const float g = in ? to_f32(gr[k].v[0]) : 0.f;
      xh[k] = in ? (to_f32(xr[k].v[0]) - m) * r : 0.f;
      ag[k] = fmaf(g, xh[k], ag[k]);
      ab[k] += g;
      wv[k] = g * (gamma && d < D ? gamma[d] : 1.f);
      s[0][0] += wv[k];
      s[1][0] = fmaf(wv[k], xh[k], s[1][0]);
    }
    if (!dx) continue;
    wave_sums<2, W, 1>(s, red[turn], w, lane);
    const float a = s[0][0] / (float)D, b = s[1][0] / (float)D;
    if (!on) continue;   // no barrier behind this
    T* dp = dx + ps.at;
#pragma unroll
    for (int k = 0; k < EPT; ++k) {
      const int d = w + W * k;
      if (d < D) dp[(long)d * inner] = from_f32<T>(r * (wv[k] - a - xh[k] * b));
    }
  }
  if (!part) return;
  float* pg = part + (size_t)blockIdx.x * D;
  float* pb = part + ((size_t)gridDim.x + blockIdx.x) * D;
#pragma unroll
  for (int k = 0; k < EPT; ++k) {
    const int d = w + W * k;
    const float tg = sum64(ag[k]), tb = sum64(ab[k]);
    if (lane == 0 && d < D) {
      pg[d] = tg;
      pb[d] = tb;
    }
  }
}

long ceil_div(long a, long b) { return (a + b - 1) / b; }

// Vectors a lane holds and waves a row takes: one wave up to 2 vectors a lane, then
// 4 waves, then 16.  On either side: one wave with 4 vectors, 16384 x 2048 bf16 backward
// 41.1 us instead of 38.8 (forward 23.3 instead of 28.7); 4 waves from 2 vectors on, 65536 x
// 512 fp32 forward 76.6 us instead of 45.8, backward 124 instead of 75; 16 waves from 16
// vectors on, 8192 x 8192 bf16 forward 55.5 us instead of 43.6, backward 80.5 instead of 81.9.
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

// Two positions a lane for 16-bit elements of an even inner axis, if the blocks still
// fill the 256 CUs (32 x 512 x 1024 bf16 forward 24.1 us against 28.7, gradients 40.4
// against 46.3).
template <typename T, typename F>
void by_positions(const NormArgs& a, F f) {
  if constexpr (sizeof(T) == 2)
    if (a.inner % 2 == 0 && a.outer * a.inner >= 256 * 128)
      return f(std::integral_constant<int, 2>());
  f(std::integral_constant<int, 1>());
}

constexpr unsigned kChBlocks = 1u << 16;   // a launch counts its threads in 32 bits

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
  // 16 waves of few channels each for 16-bit elements, 8 for fp32, whose lines fill the
  // loads (32 x 512 x 1024 with 16 against 8: bf16 24.1 against 27.8 us, fp32 35.3 against
  // 29.9; 8 x 512 x 256 bf16 10.7 against 16.6).  Above 512 channels they are
  // read again (16 x 1024 x 1024 bf16 31.6 us against 36.7 in registers; fp32 44.8
  // against 50.0).
  const unsigned n = (unsigned)(a.outer * a.inner), inner = (unsigned)a.inner;
  by_positions<T>(a, [&](auto vp) {
    constexpr int VP = decltype(vp)::value;
    const unsigned tiles = (unsigned)ceil_div(n, 64 * VP);
    const unsigned grid = tiles < kChBlocks ? tiles : kChBlocks;
#define S4_GO(ept, waves)                                                                   \
  norm_channels_kernel<T, ept, waves, VP><<<grid, 64 * waves, 0, s>>>(                      \
      x, a.gamma, a.beta, y, a.mean, a.rstd, n, D, inner, a.eps)
    constexpr int kWaves = sizeof(T) == 2 ? 16 : 8;
    if (D <= 64) S4_GO(8, 8);
    else if (D <= 256) S4_GO(256 / kWaves, kWaves);
    else if (D <= 512) S4_GO(512 / kWaves, kWaves);
    else S4_GO(0, 16);
#undef S4_GO
  });
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
    const unsigned n = (unsigned)(a.outer * a.inner), inner = (unsigned)a.inner;
    if (D <= 64) {
      norm_channels_bwd_kernel<T, 8, 8><<<dim3(nb), 512, 0, s>>>(
          x, a.gamma, a.mean, a.rstd, dy, dx, part, n, D, inner);
    } else if (D <= kNormChannels) {
      norm_channels_bwd_kernel<T, kNormChannels / 16, 16><<<dim3(nb), 1024, 0, s>>>(
          x, a.gamma, a.mean, a.rstd, dy, dx, part, n, D, inner);
    } else {
      if (dx && n > 0)
        by_positions<T>(a, [&](auto vp) {
          constexpr int VP = decltype(vp)::value;
          const unsigned tiles = (unsigned)ceil_div(n, 64 * VP);
          const unsigned grid = tiles < kChBlocks ? tiles : kChBlocks;
          norm_channels_dx_kernel<T, 16, VP><<<grid, 1024, 0, s>>>(x, a.gamma, a.mean, a.rstd, dy,
                                                                   dx, n, D, inner);
        });
      const dim3 grid((unsigned)ceil_div(D, 4 * kSums), nb);
      if (part && a.inner % Vec<T>::N == 0)
        norm_channels_sums_kernel<T, Vec<T>::N><<<grid, 256, 0, s>>>(
            x, a.mean, a.rstd, dy, part, n, D, inner);
      else if (part)
        norm_channels_sums_kernel<T, 1><<<grid, 256, 0, s>>>(x, a.mean, a.rstd, dy, part, n, D,
                                                             inner);
    }
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
