// Root-mean-square norm over rows of D contiguous values, with the residual stream's addition:
//   h = x + residual (rounded to its type: what the stream holds),
//   r = 1 / sqrt(mean_d h^2 + eps),  y = h r gamma,
// y in the type of x, or in e4m3 with a power of two as the scale of each 128 values of
// a row, or both.  Backward, with xh = h r and w = dy gamma:
//   dx = dh + r (w - xh mean_d (w xh)),  dgamma = sum dy xh,
// where dx is the gradient of x and of the residual alike.  Arithmetic is fp32, each output is
// rounded once.
//
// Both directions are bound by HBM, so a row is read once and held in registers between its sum and
// its outputs (row_shape: waves a row, both sides measured), and the next row is on its way meanwhile.
// 16384 x 4096 in bf16: forward with the residual 88 us, 6.1 TB/s, backward 122 us, 4.4 TB/s, and 5 us
// for dgamma's partial sums.
#include "fp8_device.h"
#include "norm.h"
#include "rms.h"
#include "rows_device.h"
#include "vec.h"

namespace s4 {

namespace {

// The sum over the waves of a row, in every lane; `red` is used in turn.
template <int WPR>
__device__ __forceinline__ float row_sum(float s, float (&red)[WPR]) {
  s = sum64(s);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
    __syncthreads();
    s = sum_of<WPR>(red[threadIdx.x % WPR]);
  }
  return s;
}

// Vector c .. c + VEC of a row to e4m3, and its group's scale: the 128 / VEC lanes that hold a
// group are neighbours.
template <int VEC, bool WHOLE>
__device__ __forceinline__ void store_fp8(unsigned char* __restrict__ q,
                                          unsigned char* __restrict__ scales, int D, int c,
                                          const float* v) {
  unsigned big = 0;
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const unsigned m = c + j < D ? magnitude(v[j]) : 0u;
    big = m > big ? m : big;
  }
  const unsigned byte = scale_byte(max_of<kGroup / VEC>(big));
  const float f = inverse_scale(byte);
  unsigned t[VEC / 4];
#pragma unroll
  for (int j = 0; j < VEC; j += 4)
    t[j / 4] = pack4(v[j] * f, v[j + 1] * f, v[j + 2] * f, v[j + 3] * f);
  if (c + VEC <= D) {
    __builtin_memcpy(q + c, t, VEC);
  } else if constexpr (!WHOLE) {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (c + j < D) q[c + j] = (unsigned char)(t[j / 4] >> (8 * (j % 4)));
  }
  if (c % kGroup == 0 && c < D) scales[c / kGroup] = (unsigned char)byte;
}

}  // namespace

// WPR waves share a row (blocks of 256 threads hold 4 rows at WPR = 1), and a block walks over
// rows blockIdx, blockIdx + gridDim, ..., the next row on its way while one is computed.
template <typename T, int NV, int WPR, bool WHOLE>
__global__ __launch_bounds__(WPR > 4 ? 64 * WPR : kRowThreads) void rms_rows_kernel(
    const T* x, const T* residual, const float* __restrict__ gamma, T* h, T* y,
    unsigned char* __restrict__ q, unsigned char* __restrict__ scales, float* __restrict__ rstd,
    long rows, int D, float eps) {
  using Part = RowPart<T, NV, WPR, WHOLE>;
  using One = RowPart<T, 1, WPR, WHOLE>;
  constexpr int VEC = Part::VEC, E = Part::E;
  constexpr int RPB = WPR == 1 ? kRowThreads / 64 : 1;
  __shared__ float red[2][WPR];
  const int tid = WPR == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int groups = (D + kGroup - 1) / kGroup;
  long row = (long)blockIdx.x * RPB + (WPR == 1 ? w : 0);
  if (row >= rows) return;   // WPR > 1: the whole block
  Part next, nres;
  next.load(x + row * D, D, tid);
  if (residual) nres.load(residual + row * D, D, tid);
  constexpr bool kWide = wide_rows(E, WPR);
  float gm[kWide ? 1 : E];
  if constexpr (!kWide) Part::columns(gamma, D, tid, 1.f, gm);
  int turn = 0;
  for (; row < rows; turn ^= 1) {
    float v[E];
    next.get(D, tid, v);
    if (residual) {
      float u[E];
      nres.get(D, tid, u);
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = to_f32(from_f32<T>(v[i] + u[i]));
    }
    const long here = row;
    row += (long)gridDim.x * RPB;
    if (row < rows) {
      next.load(x + row * D, D, tid);
      if (residual) nres.load(residual + row * D, D, tid);
    }
    if (h) Part::store(h + here * D, D, tid, v);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(v[i], v[i], s);   // behind D: 0
    s = row_sum<WPR>(s, red[turn]);
    const float r = 1.f / sqrtf(s / (float)D + eps);
    T* yr = y ? y + here * D : nullptr;
    unsigned char* qr = q ? q + here * D : nullptr;
    unsigned char* sr = q ? scales + here * groups : nullptr;
    const int t0 = kWide ? opaque(tid) : tid;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float* u = v + i * VEC;
      if constexpr (kWide) {
        float g[VEC];
        One::columns(gamma, D, t0 + i * WPR * 64, 1.f, g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) u[j] = u[j] * r * g[j];
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) u[j] = u[j] * r * gm[i * VEC + j];
      }
      if (y) One::store(yr, D, t0 + i * WPR * 64, u);
      if (q) store_fp8<VEC, WHOLE>(qr, sr, D, One::at(0, t0 + i * WPR * 64), u);
    }
    if (tid == 0 && rstd) rstd[here] = r;
  }
}

// Every lane keeps the same columns of all its block's rows, so dgamma's sums stay in its
// registers and leave the block once, as row blockIdx of part [gridDim][D].
template <typename T, int NV, int WPR, bool WHOLE>
__global__ __launch_bounds__(WPR > 4 ? 64 * WPR : kRowThreads) void rms_rows_bwd_kernel(
    const T* __restrict__ h, const float* __restrict__ gamma, const float* __restrict__ rstd,
    const T* __restrict__ dy, const T* dh, T* dx, float* __restrict__ part, long rows, int D) {
  using Part = RowPart<T, NV, WPR, WHOLE>;
  constexpr int VEC = Part::VEC, E = Part::E;
  constexpr int RPB = WPR == 1 ? kRowThreads / 64 : 1;
  __shared__ float red[2][WPR];
  __shared__ float cols[WPR == 1 ? 3 * 64 * E : 1];
  const int tid = WPR == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int sub = WPR == 1 ? threadIdx.x >> 6 : 0;
  float gm[E], ag[E];
  Part nx, ng;
  float nr = 0.f;
  long row = (long)blockIdx.x * RPB + sub;
  if (row < rows) {
    nx.load(h + row * D, D, tid);
    ng.load(dy + row * D, D, tid);
    nr = rstd[row];
  }
  Part::columns(gamma, D, tid, 1.f, gm);
#pragma unroll
  for (int i = 0; i < E; ++i) ag[i] = 0.f;
  int turn = 0;
  for (; row < rows; turn ^= 1) {
    float xv[E], gv[E];
    nx.get(D, tid, xv);
    ng.get(D, tid, gv);
    const float r = nr;
    const long here = row;
    Part nd;   // needed last
    if (dx && dh) nd.load(dh + here * D, D, tid);
    row += (long)gridDim.x * RPB;
    if (row < rows) {
      nx.load(h + row * D, D, tid);
      ng.load(dy + row * D, D, tid);
      nr = rstd[row];
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      // behind D, dy = 0: nothing is added
      const float xh = xv[i] * r, w = gv[i] * gm[i];
      xv[i] = xh;
      s = fmaf(w, xh, s);
      ag[i] = fmaf(gv[i], xh, ag[i]);
      gv[i] = w;
    }
    if (dx) {
      s = row_sum<WPR>(s, red[turn]) / (float)D;
#pragma unroll
      for (int i = 0; i < E; ++i) gv[i] = r * (gv[i] - xv[i] * s);
      if (dh) {
        nd.get(D, tid, xv);
#pragma unroll
        for (int i = 0; i < E; ++i) gv[i] += xv[i];
      }
      Part::store(dx + here * D, D, tid, gv);
    }
  }
  if (!part) return;
  float* pg = part + (size_t)blockIdx.x * D;
  if constexpr (WPR == 1) {   // the four waves hold the same columns
    if (sub)
#pragma unroll
      for (int i = 0; i < E; ++i) cols[((sub - 1) * E + i) * 64 + tid] = ag[i];
    __syncthreads();
    if (sub) return;
#pragma unroll
    for (int i = 0; i < E; ++i)
      ag[i] += (cols[i * 64 + tid] + cols[(E + i) * 64 + tid]) + cols[(2 * E + i) * 64 + tid];
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = Part::at(i, tid);
    if (c + VEC <= D) {
      __builtin_memcpy(pg + c, ag + i * VEC, VEC * sizeof(float));
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (c + j < D) pg[c + j] = ag[i * VEC + j];
    }
  }
}

// Backward over wide rows, in two kernels, since a row's columns leave no registers for
// their sums: dx by rows (h and dy are read again behind the row's sum, from the caches), and
// the columns' sums.
template <typename T, int WPR, bool WHOLE>
__global__ __launch_bounds__(64 * WPR) void rms_wide_dx_kernel(
    const T* __restrict__ h, const float* __restrict__ gamma, const float* __restrict__ rstd,
    const T* __restrict__ dy, const T* dh, T* dx, long rows, int D) {
  using One = RowPart<T, 1, WPR, WHOLE>;
  constexpr int VEC = One::VEC, STEP = 64 * WPR;
  __shared__ float red[2][WPR];
  const int tid = threadIdx.x;
  int turn = 0;
  for (long row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
    const T *hr = h + row * D, *gr = dy + row * D;
    const float r = rstd[row];
    auto vectors = [&](auto f) {   // f(at, xh, dy gamma); a whole step is inside or partly
      One xo, go;
      float xv[VEC], gv[VEC], g[VEC];
#pragma unroll 2
      for (int at = tid; at * VEC < D; at += STEP) {
        xo.load(hr, D, at);
        go.load(gr, D, at);
        One::columns(gamma, D, at, 1.f, g);
        xo.get(D, at, xv);
        go.get(D, at, gv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          xv[j] *= r;
          gv[j] *= g[j];
        }
        f(at, xv, gv);
      }
    };
    float s = 0.f;
    vectors([&](int, const float* xh, const float* w) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) s = fmaf(w[j], xh[j], s);   // behind D, w = 0
    });
    s = row_sum<WPR>(s, red[turn]) / (float)D;
    vectors([&](int at, const float* xh, const float* w) {
      float o[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = r * (w[j] - xh[j] * s);
      if (dh) {
        One d;
        float dv[VEC];
        d.load(dh + row * D, D, at);
        d.get(D, at, dv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] += dv[j];
      }
      One::store(dx + row * D, D, at, o);
    });
  }
}

// Block: 64 vectors of columns, the rows blockIdx.y 4 + wave and on by gridDim.y 4.
template <typename T, bool WHOLE>
__global__ __launch_bounds__(256) void rms_wide_sums_kernel(
    const T* __restrict__ h, const float* __restrict__ rstd, const T* __restrict__ dy,
    float* __restrict__ part, long rows, int D) {
  using One = RowPart<T, 1, 1, WHOLE>;
  constexpr int VEC = One::VEC;
  __shared__ float red[3][VEC][64];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int at = blockIdx.x * 64 + lane;
  float ag[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) ag[j] = 0.f;
#pragma unroll 4
  for (long row = blockIdx.y * 4 + w; row < rows; row += gridDim.y * 4) {
    One xo, go;
    float xv[VEC], gv[VEC];
    xo.load(h + row * D, D, at);
    go.load(dy + row * D, D, at);
    const float r = rstd[row];
    xo.get(D, at, xv);
    go.get(D, at, gv);
#pragma unroll
    for (int j = 0; j < VEC; ++j) ag[j] = fmaf(gv[j], xv[j] * r, ag[j]);
  }
  if (w > 0)
#pragma unroll
    for (int j = 0; j < VEC; ++j) red[w - 1][j][lane] = ag[j];
  __syncthreads();
  if (w > 0) return;
  float* pg = part + (size_t)blockIdx.y * D;
#pragma unroll
  for (int j = 0; j < VEC; ++j)
    if (at * VEC + j < D)
      pg[at * VEC + j] = ag[j] + ((red[0][j][lane] + red[1][j][lane]) + red[2][j][lane]);
}

namespace {

template <typename T>
hipError_t fwd(const RmsArgs& a, hipStream_t s) {
  const int D = (int)a.D;
  row_shape<T>(D, [&](auto nv, auto wpr, auto whole) {
    constexpr int NV = decltype(nv)::value, WPR = decltype(wpr)::value;
    constexpr bool W = decltype(whole)::value;
    const long blocks = WPR == 1 ? ceil_div(a.rows, kRowThreads / 64) : a.rows;
    const long most = WPR > 4 ? kNormBlocks / 4 : kNormBlocks;
    rms_rows_kernel<T, NV, WPR, W>
        <<<dim3((unsigned)(blocks < most ? blocks : most)), WPR > 4 ? 64 * WPR : kRowThreads, 0,
           s>>>((const T*)a.x, (const T*)a.residual, a.gamma, (T*)a.h, (T*)a.y, a.q, a.scales,
                a.rstd, a.rows, D, a.eps);
  });
  return hipGetLastError();
}

template <typename T>
hipError_t bwd(const RmsArgs& a, hipStream_t s) {
  const T *h = (const T*)a.x, *dy = (const T*)a.dy, *dh = (const T*)a.dh;
  T* dx = (T*)a.dx;
  const int D = (int)a.D, nb = (int)norm_parts(a.rows, a.D, 1);
  float* part = a.dgamma ? a.part : nullptr;
  row_shape<T>(D, [&](auto nv, auto wpr, auto whole) {
    constexpr int NV = decltype(nv)::value, WPR = decltype(wpr)::value;
    constexpr bool W = decltype(whole)::value;
    if constexpr (wide_rows(NV * Vec<T>::N, WPR)) {
      if (dx && a.rows > 0)
        rms_wide_dx_kernel<T, WPR, W><<<dim3((unsigned)(a.rows < 512 ? a.rows : 512)), 64 * WPR, 0, s>>>(
            h, a.gamma, a.rstd, dy, dh, dx, a.rows, D);
      if (part)
        rms_wide_sums_kernel<T, W><<<dim3((unsigned)ceil_div(D, 64 * Vec<T>::N), nb), 256, 0, s>>>(
            h, a.rstd, dy, part, a.rows, D);
    } else {
      rms_rows_bwd_kernel<T, NV, WPR, W><<<dim3(nb), WPR > 4 ? 64 * WPR : kRowThreads, 0, s>>>(
          h, a.gamma, a.rstd, dy, dh, dx, part, a.rows, D);
    }
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !part) return e;
  return launch_columns(part, nb, D, a.dgamma, nullptr, s);
}

}  // namespace

hipError_t launch_rms_fwd(const RmsArgs& a, int dtype, hipStream_t s) {
  return dtype == S4DPLR_F32 ? fwd<float>(a, s) : dtype == S4DPLR_BF16 ? fwd<bf16>(a, s) : fwd<f16>(a, s);
}

hipError_t launch_rms_bwd(const RmsArgs& a, int dtype, hipStream_t s) {
  return dtype == S4DPLR_F32 ? bwd<float>(a, s) : dtype == S4DPLR_BF16 ? bwd<bf16>(a, s) : bwd<f16>(a, s);
}

}  // namespace s4
