// Gated delta rule, token by token: the serving form.  With p = S^T k, z = S^T q
// (S before the token),
//   n = v - a p,  o = scale (a z + (q . k) beta n),  S <- a S + k (beta n)^T,
// so one pass over the state and one sum across its rows give a token.  A block
// of 256 threads holds kCols columns of one head's state in registers (8 lanes x
// 4 columns, 32 groups of rows), so a head is spread over dv / 32 blocks and a row of 32
// columns is a whole line; for one token the state's read and write bound it (128
// sequences of 16 heads of 128 x 128: 52 us, 5.2 TB/s).
#include "delta_device.h"

namespace s4 {

namespace {
constexpr int kCols = 32, kGroups = 32;
}

template <typename T, int RPG>   // rows of the state per thread: dk <= 32 RPG
__global__ __launch_bounds__(256) void delta_step_kernel(const s4dplr_delta_plan p,
                                                         const DeltaArgs a) {
  __shared__ float qs[2][32 * RPG], ks[2][32 * RPG];
  __shared__ __attribute__((aligned(16))) float red[2][4][2][kCols];
  __shared__ float qk[2][4];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  int sh, slice;
  if (!slice_of(p.sequences * p.Hv, (p.dv + kCols - 1) / kCols, &sh, &slice)) return;
  const int s = sh / p.Hv, h = sh % p.Hv, hk = h / (p.Hv / p.Hk);
  const Rows r = rows_of(p, a.offsets, s);
  if (r.len > a.step_tokens) return;
  const int col = slice * kCols + 4 * (lane & 7), g = w * 8 + (lane >> 3);
  const int m = p.dv - col;   // columns of this lane: 4 or fewer
  v4f S[RPG];
#pragma unroll
  for (int i = 0; i < RPG; ++i) {
    const int d = g + kGroups * i;
    S[i] = v4f{0.f, 0.f, 0.f, 0.f};
    if (a.state && d < p.dk) {
      const float* sp = a.state + ((size_t)sh * p.dk + d) * p.dv + col;
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
    for (int d = tid; d < p.dk; d += 256) {
      qs[b][d] = to_f32(((const T*)a.q)[at * a.ldq + (size_t)hk * p.dk + d]);
      ks[b][d] = to_f32(((const T*)a.k)[at * a.ldk + (size_t)hk * p.dk + d]);
    }
    const float decay = expf(a.g[at * p.Hv + h]), beta = a.beta[at * p.Hv + h];
    v4f v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < m) v[e] = to_f32(((const T*)a.v)[at * a.ldv + (size_t)h * p.dv + col + e]);
    __syncthreads();
    v4f pk = {0.f, 0.f, 0.f, 0.f}, pq = pk;
    float kv[RPG], dot = 0.f;
#pragma unroll
    for (int i = 0; i < RPG; ++i) {
      const int d = g + kGroups * i;
      const float q = d < p.dk ? qs[b][d] : 0.f;
      kv[i] = d < p.dk ? ks[b][d] : 0.f;
      pk += S[i] * kv[i];
      pq += S[i] * q;
      dot = fmaf(q, kv[i], dot);
    }
#pragma unroll
    for (int off = 8; off < 64; off <<= 1) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        pk[e] += __shfl_xor(pk[e], off);
        pq[e] += __shfl_xor(pq[e], off);
      }
      dot += __shfl_xor(dot, off);
    }
    if (lane < 8) {
      *reinterpret_cast<v4f*>(&red[b][w][0][4 * lane]) = pk;
      *reinterpret_cast<v4f*>(&red[b][w][1][4 * lane]) = pq;
      if (lane == 0) qk[b][w] = dot;
    }
    __syncthreads();
    pk = pq = v4f{0.f, 0.f, 0.f, 0.f};
    dot = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      pk += *reinterpret_cast<const v4f*>(&red[b][i][0][4 * (lane & 7)]);
      pq += *reinterpret_cast<const v4f*>(&red[b][i][1][4 * (lane & 7)]);
      dot += qk[b][i];
    }
    const v4f u = (v - pk * decay) * beta;
#pragma unroll
    for (int i = 0; i < RPG; ++i) S[i] = S[i] * decay + u * kv[i];
    if (g == 0) {
      const v4f o = (pq * decay + u * dot) * a.scale;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < m) ((T*)a.o)[(at * p.Hv + h) * p.dv + col + e] = from_f32<T>(o[e]);
    }
  }
  if (!a.state_out) return;
#pragma unroll
  for (int i = 0; i < RPG; ++i) {
    const int d = g + kGroups * i;
    if (d < p.dk) {
      float* sp = a.state_out + ((size_t)sh * p.dk + d) * p.dv + col;
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
hipError_t steps(const s4dplr_delta_plan* p, const DeltaArgs& a, hipStream_t s) {
  const unsigned heads = (unsigned)(p->sequences * p->Hv);
  const unsigned grid = (heads + 7) / 8 * 8 * ((p->dv + kCols - 1) / kCols);
  if (p->dk <= 64) delta_step_kernel<T, 2><<<grid, 256, 0, s>>>(*p, a);
  else if (p->dk <= 128) delta_step_kernel<T, 4><<<grid, 256, 0, s>>>(*p, a);
  else delta_step_kernel<T, 8><<<grid, 256, 0, s>>>(*p, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_steps(const s4dplr_delta_plan* p, const DeltaArgs& a, hipStream_t s) {
  if (p->dtype == S4DPLR_F32) return steps<float>(p, a, s);
  if (p->dtype == S4DPLR_BF16) return steps<bf16>(p, a, s);
  return steps<f16>(p, a, s);
}

}  // namespace s4
