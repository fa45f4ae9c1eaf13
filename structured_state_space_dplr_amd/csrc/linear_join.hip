// Linear attention: what joins the blocks of a pass.  The states before the segments from what
// the segments add, the gradients of shared heads, and the gradient of the decays.
#include "linear_device.h"

namespace s4 {

namespace {

// Per sequence of several segments and head, element by element: from the state before the first
// segment (rev: behind the last), slot m takes the state before segment m (behind it),
//   run <- decay_m run + added_m.
// Bound by the states' read and write: 32 segments of 16 heads of 128 x 128 15 us, 4.5 TB/s.  Eight
// slots' loads are on their way together.
// V: elements a lane, 4 where a state is a multiple of them.
template <int V>
__global__ __launch_bounds__(256) void linear_scan_kernel(const LinPass p) {
  typedef float Vf __attribute__((ext_vector_type(V)));
  const int s = blockIdx.x / p.Hv, h = blockIdx.x % p.Hv;
  const LinRows r = lin_rows(p, s);
  if (r.len <= p.segment) return;
  const long sz = (long)p.dk * p.dv, at = ((long)blockIdx.y * 256 + threadIdx.x) * V;
  if (at >= sz) return;
  const long base = r.slot(s, p.segment);
  int n = r.segments(p.segment);
  if (base + n > p.slots) n = (int)(p.slots - base);
  Vf run = {};
  if (p.first) __builtin_memcpy(&run, p.first + ((size_t)s * p.Hv + h) * sz + at, sizeof(run));
  constexpr int AHEAD = 8;
  for (int m0 = 0; m0 < n; m0 += AHEAD) {
    Vf add[AHEAD];
    float dec[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int m = m0 + i < n ? m0 + i : n - 1;
      const size_t slot = (size_t)(base + (p.rev ? n - 1 - m : m)) * p.Hv + h;
      __builtin_memcpy(&add[i], p.states + slot * sz + at, sizeof(Vf));
      dec[i] = p.decay[slot];
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float v = add[i][e];
        touch(v);
        add[i][e] = v;
      }
      touch(dec[i]);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int m = m0 + i;
      if (m >= n) break;
      const size_t slot = (size_t)(base + (p.rev ? n - 1 - m : m)) * p.Hv + h;
      __builtin_memcpy(p.states + slot * sz + at, &run, sizeof(Vf));
#pragma unroll
      for (int e = 0; e < V; ++e) run[e] = fmaf(dec[i], run[e], add[i][e]);   // behind the last: not used
    }
  }
}

// Both gradients of a call in one launch, one of blockIdx.y each.
template <typename T>
__global__ __launch_bounds__(256) void linear_groups_kernel(const LinGroups a) {
  const float* __restrict__ part = a.part[blockIdx.y];
  T* __restrict__ out = (T*)a.out[blockIdx.y];
  if (!out) return;
  const int Hk = a.Hk, group = a.Hv / a.Hk, d = a.d;
  // the rows of the sequences, which lie one behind the other
  long lo = 0, hi = a.tokens;
  if (a.offsets) {
    const Rows r = clamp_rows((int)a.tokens, a.offsets[0], a.offsets[a.sequences]);
    lo = r.start;
    hi = r.start + r.len;
  }
  const long n = hi * Hk * d;
  for (long at = lo * Hk * d + (long)blockIdx.x * 256 + threadIdx.x; at < n; at += (long)gridDim.x * 256) {
    const long row = at / d, c = at % d;   // row: token and key head
    const float* from = part + row * group * d + c;
    float s = from[0];
    for (int i = 1; i < group; ++i) s += from[(long)i * d];
    out[at] = from_f32<T>(s);
  }
}

// dg_t = <S_{t-1}, gradient of S_{t-1} by what comes later>: the edge before the segment, and
// behind token i  + k_i . dk_i - q_i . dq_i  of the token itself.  The sums are held in 64 bits
// over a segment of a few hundred tokens.  A block per segment and head, 64 tokens a wave; all parts
// of a token are loaded together (4 x 4096 tokens of 16 heads, 17 MB: 25 us one by one, 15 so).
// Where exp(g) is 0 nothing of the state before is left, and dg is 0.
__global__ __launch_bounds__(512) void linear_gates_kernel(const LinGates a) {
  __shared__ double sums[2][8], totals[8];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = blockIdx.y;
  LinItem it;
  const long skip = a.offsets || a.each <= a.segment ? 0 : a.sequences;
  const long item = skip + blockIdx.x;
  if (!lin_item(a, item, &it)) {
    if (threadIdx.x == 0 && a.ldg == 0) a.sums[item * a.Hv + h] = 0.f;
    return;
  }
  double run = 0.0, total = 0.0;
  if (it.len > 0) {
    const float e = lane < a.parts_edge ? a.edge[(item * a.Hv + h) * kDotParts + lane] : 0.f;
    run = e;
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) run += __shfl_xor(run, off);
    run = __shfl(run, 0);
  }
  int turn = 0;
  for (int t0 = 64 * w; t0 - 64 * w < it.len; t0 += 512, turn ^= 1) {
    const bool in = t0 + lane < it.len;
    const long tok = it.start + (in ? t0 + lane : 0);
    const float *kp = a.dotk + (size_t)h * a.tokens + tok, *qp = a.dots + (size_t)h * a.tokens + tok;
    const size_t step = (size_t)a.Hv * a.tokens;
    float dk[kDotParts], dq[kDotParts];
#pragma unroll
    for (int i = 0; i < kDotParts; ++i) {
      dk[i] = kp[(i < a.parts_k ? i : 0) * step];
      dq[i] = qp[(i < a.parts_q ? i : 0) * step];
    }
    const float g = a.g[tok * a.ldg + h];
    double own = 0.0;
#pragma unroll
    for (int i = 0; i < kDotParts; ++i) {
      touch(dk[i]);
      touch(dq[i]);
    }
#pragma unroll
    for (int i = 0; i < kDotParts; ++i) {
      if (i < a.parts_k) own += dk[i];
      if (i < a.parts_q) own -= dq[i];
    }
    own = in ? own : 0.0;
    double x = own;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const double y = __shfl_up(x, off);
      if (lane >= off) x += y;
    }
    if (lane == 63) sums[turn][w] = x;
    __syncthreads();
    double before = run;   // of the waves before this one
    for (int i = 0; i < 8; ++i) {
      const double y = sums[turn][i];
      if (i < w) before += y;
      run += y;
    }
    const double dg = expf(g) == 0.f ? 0.0 : before + (x - own);
    if (in && a.ldg) a.dg[tok * a.Hv + h] = (float)dg;
    total += in ? dg : 0.0;
  }
  if (a.ldg == 0) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) total += __shfl_xor(total, off);
    if (lane == 0) totals[w] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < 8; ++i) total += totals[i];
      a.sums[item * a.Hv + h] = (float)total;
    }
  }
}

// dg of one decay a head: the items' sums, always in the same order.
__global__ __launch_bounds__(256) void linear_gate_sums_kernel(const float* __restrict__ sums,
                                                               long first, long last, int Hv,
                                                               float* __restrict__ dg) {
  __shared__ double red[256];
  const int h = blockIdx.x;
  double s = 0.0;
  for (long i = first + threadIdx.x; i < last; i += 256) s += sums[i * Hv + h];
  red[threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.x >= 64) return;
  s = (red[threadIdx.x] + red[threadIdx.x + 64]) + (red[threadIdx.x + 128] + red[threadIdx.x + 192]);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off);
  if (threadIdx.x == 0) dg[h] = (float)s;
}

}  // namespace

hipError_t linear_pass_bf16(const LinPass& a, bool sum, hipStream_t s);
hipError_t linear_pass_f16(const LinPass& a, bool sum, hipStream_t s);
hipError_t linear_pass_f32(const LinPass& a, bool sum, hipStream_t s);
int linear_parts_bf16(int dx, int dw);
int linear_parts_f16(int dx, int dw);
int linear_parts_f32(int dx, int dw);

namespace {
hipError_t pass(const LinPass& a, bool sum, int dtype, hipStream_t s) {
  return dtype == S4DPLR_F32 ? linear_pass_f32(a, sum, s)
         : dtype == S4DPLR_BF16 ? linear_pass_bf16(a, sum, s) : linear_pass_f16(a, sum, s);
}
}  // namespace

int linear_parts(int dx, int dw, int dtype) {
  return dtype == S4DPLR_F32 ? linear_parts_f32(dx, dw)
         : dtype == S4DPLR_BF16 ? linear_parts_bf16(dx, dw) : linear_parts_f16(dx, dw);
}

hipError_t launch_linear_pass(const LinPass& a, int dtype, hipStream_t s) {
  return pass(a, false, dtype, s);
}

hipError_t launch_linear_sums(const LinPass& a, int dtype, hipStream_t s) {
  if (a.slots == 0 || (!a.offsets && a.each <= a.segment)) return hipSuccess;   // one segment each
  const hipError_t e = pass(a, true, dtype, s);
  if (e != hipSuccess) return e;
  const long sz = (long)a.dk * a.dv;
  const unsigned heads = (unsigned)(a.sequences * a.Hv);
  if (sz % 4 == 0)
    linear_scan_kernel<4><<<dim3(heads, (unsigned)((sz + 1023) / 1024)), 256, 0, s>>>(a);
  else
    linear_scan_kernel<1><<<dim3(heads, (unsigned)((sz + 255) / 256)), 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_linear_groups(const LinGroups& a, int dtype, hipStream_t s) {
  const long n = a.tokens * a.Hk * a.d;
  if (n == 0) return hipSuccess;
  const long blocks = (n + 255) / 256;
  const dim3 grid((unsigned)(blocks < (1 << 16) ? blocks : 1 << 16), 2);
  if (dtype == S4DPLR_F32) linear_groups_kernel<float><<<grid, 256, 0, s>>>(a);
  else if (dtype == S4DPLR_BF16) linear_groups_kernel<bf16><<<grid, 256, 0, s>>>(a);
  else linear_groups_kernel<f16><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_linear_gates(const LinGates& a, hipStream_t s) {
  const bool all_long = !a.offsets && a.each > a.segment, all_short = !a.offsets && !all_long;
  const long first = all_long ? a.sequences : 0, last = all_short ? a.sequences : a.sequences + a.slots;
  if (last > first)
    linear_gates_kernel<<<dim3((unsigned)(last - first), (unsigned)a.Hv), 512, 0, s>>>(a);
  if (a.ldg == 0)
    linear_gate_sums_kernel<<<dim3((unsigned)a.Hv), 256, 0, s>>>(a.sums, first, last, a.Hv, a.dg);
  return hipGetLastError();
}

}  // namespace s4
