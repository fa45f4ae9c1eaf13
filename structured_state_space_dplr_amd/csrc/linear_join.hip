// Linear attention: what joins the blocks of a pass.  The states before the segments from what
// the segments add, and the gradients of shared heads.
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

}  // namespace s4
