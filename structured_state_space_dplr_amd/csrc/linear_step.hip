// Linear attention, token by token: the serving form,
//   S <- exp(g) S + k v^T,  o = scale S^T q,
// one pass over the state a token.  A block of 256 threads holds kCols columns of one head's state
// in registers (8 lanes x 4 columns, 32 groups of rows), so a head is spread over dv / 32 blocks
// and a row of 32 columns is a whole line; for one token the state's read and write bound it (128
// sequences of 16 heads of 128 x 128: 53 us, 5.1 TB/s; one sequence of 16 heads of 64 x 64: 3.7).
#include "linear_device.h"

namespace s4 {

namespace {
constexpr int kCols = 32, kGroups = 32;
}

template <typename T, int RPG>   // rows of the state per thread: dk <= 32 RPG
__global__ __launch_bounds__(256) void linear_step_kernel(const LinStep a) {
  __shared__ float qs[2][32 * RPG], ks[2][32 * RPG];
  __shared__ __attribute__((aligned(16))) float red[2][4][kCols];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  int sh, slice;
  if (!slice_of(a.sequences * a.Hv, (a.dv + kCols - 1) / kCols, &sh, &slice)) return;
  const int s = sh / a.Hv, h = sh % a.Hv, hk = h / (a.Hv / a.Hk);
  const LinRows r = lin_rows(a, s);
  if (r.len > a.step_tokens) return;
  const int col = slice * kCols + 4 * (lane & 7), g = w * 8 + (lane >> 3);
  const int m = a.dv - col;   // columns of this lane: 4 or fewer
  v4f S[RPG];
#pragma unroll
  for (int i = 0; i < RPG; ++i) {
    const int d = g + kGroups * i;
    S[i] = v4f{0.f, 0.f, 0.f, 0.f};
    if (a.state && d < a.dk) {
      const float* sp = a.state + ((size_t)sh * a.dk + d) * a.dv + col;
      if (m >= 4) __builtin_memcpy(&S[i], sp, 16);
      else
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (e < m) S[i][e] = sp[e];
    }
  }
  for (long t = 0; t < r.len; ++t) {
    const int b = (int)(t & 1);
    const long at = r.start + t;
    for (int d = tid; d < a.dk; d += 256) {
      qs[b][d] = to_f32(((const T*)a.q)[at * a.ldq + (size_t)hk * a.dk + d]);
      ks[b][d] = to_f32(((const T*)a.k)[at * a.ldk + (size_t)hk * a.dk + d]);
    }
    const float decay = a.g ? expf(a.g[at * a.ldg + h]) : 1.f;
    v4f v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < m) v[e] = to_f32(((const T*)a.v)[at * a.ldv + (size_t)h * a.dv + col + e]);
    __syncthreads();
    v4f o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < RPG; ++i) {
      const int d = g + kGroups * i;
      const float q = d < a.dk ? qs[b][d] : 0.f, k = d < a.dk ? ks[b][d] : 0.f;
      S[i] = S[i] * decay + v * k;
      o += S[i] * q;
    }
#pragma unroll
    for (int off = 8; off < 64; off <<= 1)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], off);
    if (lane < 8) *reinterpret_cast<v4f*>(&red[b][w][4 * lane]) = o;
    __syncthreads();
    if (g == 0) {
      o = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i) o += *reinterpret_cast<const v4f*>(&red[b][i][4 * (lane & 7)]);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < m) ((T*)a.o)[(at * a.Hv + h) * a.dv + col + e] = from_f32<T>(o[e] * a.scale);
    }
  }
  if (!a.state_out) return;
#pragma unroll
  for (int i = 0; i < RPG; ++i) {
    const int d = g + kGroups * i;
    if (d < a.dk) {
      float* sp = a.state_out + ((size_t)sh * a.dk + d) * a.dv + col;
      if (m >= 4) __builtin_memcpy(sp, &S[i], 16);
      else
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (e < m) sp[e] = S[i][e];
    }
  }
}

namespace {

template <typename T>
hipError_t steps(const LinStep& a, hipStream_t s) {
  const unsigned heads = (unsigned)(a.sequences * a.Hv);
  const unsigned grid = (heads + 7) / 8 * 8 * ((a.dv + kCols - 1) / kCols);
  if (a.dk <= 64) linear_step_kernel<T, 2><<<grid, 256, 0, s>>>(a);
  else if (a.dk <= 128) linear_step_kernel<T, 4><<<grid, 256, 0, s>>>(a);
  else linear_step_kernel<T, 8><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_steps(const LinStep& a, int dtype, hipStream_t s) {
  if (dtype == S4DPLR_F32) return steps<float>(a, s);
  if (dtype == S4DPLR_BF16) return steps<bf16>(a, s);
  return steps<f16>(a, s);
}

}  // namespace s4
