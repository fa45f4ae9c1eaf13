// Linear attention: the gradient of the decays.  Per value head, with a_t = exp(g_t), G the inclusive sums
// of g, and Z behind row i the gradient of the state there by what comes later,
//   dg_t = a_t <S_{t-1}, gradient of S_t> = sum over the pairs i < t <= j of
//          x_ij = scale (q_j . k_i) (do_j . v_i) exp(G_j - G_i),
// where the state before the first row stands for the rows before it and the gradient of the last state for
// those behind it.  Over a chunk of rows 1 .. C, with S before and Z behind it:
//   dg_t = sum_{i < t <= j} x_ij + sum_{j >= t} b_j + sum_{i < t} c_i + exp(G_C) <S, Z>,
//   b_j = scale exp(G_j) q_j^T S do_j,   c_i = exp(G_C - G_i) k_i^T Z v_i.
// Every term straddles t, so dg_t is off by the rounding of what it consists of, however fast a head
// forgets: running sums of k . dk - q . dq would be cheaper, and carry the rounding of slow tokens' sums,
// and of each token's own q . k, to tokens whose decay has made dg smaller than that.
//
// The passes for dq and dk leave b, c and (in place of c_C) the last term, each by parts of the columns
// (LinPass::dot).  The pairs inside the chunk are summed here, both products on the bf16 matrix cores: a block
// has a chunk of a head, a wave a strip of 16 rows j.  4 x 4096 tokens of 16 heads of 128 x 128 in bf16: 69
// us for 302 MB, 4.4 TB/s (operands straight from memory, without LDS: 320).
#include "linear_device.h"

namespace s4 {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

// C rows of a tensor's head, 128 bytes of each a step, on their way to LDS: 16-byte piece p of row r lies at
// p ^ (r % 8), so that 16 rows of one piece do not share banks.
template <typename T, int C, bool WHOLE>
struct GateTile {
  static constexpr int VEC = 16 / (int)sizeof(T), THREADS = 4 * C, N = C * 8 / THREADS;
  static constexpr int BYTES = C * 128;
  T v[N][VEC];
  // columns c0 and on of the n rows from `base` on, ld elements apart; rows behind the end: the last one,
  // whose pairs are left out
  __device__ __forceinline__ void fetch(const unsigned char* __restrict__ base, unsigned ld, int n, int c0, int d) {
    const unsigned tid = thread();
    const int col = c0 + (int)(tid & 7) * VEC;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = (int)(tid >> 3) + i * (THREADS / 8);
      const unsigned at = (unsigned)(r < n ? r : n - 1) * (ld * (unsigned)sizeof(T));
      if constexpr (WHOLE) {
        __builtin_memcpy(v[i], base + (at + (col < d ? col : 0) * (unsigned)sizeof(T)), 16);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          __builtin_memcpy(&v[i][j], base + (at + (col + j < d ? col + j : 0) * (unsigned)sizeof(T)), sizeof(T));
      }
    }
  }
  __device__ __forceinline__ void stage(unsigned char* to, int c0, int d) const {
    const unsigned tid = thread();
    const int p = tid & 7, col = c0 + p * VEC;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = (int)(tid >> 3) + i * (THREADS / 8);
      T t[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) t[j] = col + (WHOLE ? 0 : j) < d ? v[i][j] : (T)0.f;
      v4i x;
      __builtin_memcpy(&x, t, 16);
      *reinterpret_cast<v4i*>(to + r * 128 + (p ^ (r & 7)) * 16) = x;
    }
  }
};
// Operand: columns 32 ks + 8 (lane / 16) and on of row `strip` 16 + lane % 16.
template <typename T, int PARTS>
__device__ __forceinline__ void gate_operand(const unsigned char* m, int strip, int ks, v8bf (&out)[PARTS]) {
  const unsigned tid = thread();
  const int r = 16 * strip + (tid & 15), lg = (tid & 63) >> 4;
  if constexpr (sizeof(T) == 2) {
    const v4i x = *reinterpret_cast<const v4i*>(m + r * 128 + ((4 * ks + lg) ^ (r & 7)) * 16);
    if constexpr (PARTS == 1) {
      __builtin_memcpy(&out[0], &x, 16);
    } else {
      T t[8];
      float f[8];
      __builtin_memcpy(t, &x, 16);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = to_f32(t[j]);
      split8<PARTS>(f, out);
    }
  } else {
    float f[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const v4i x = *reinterpret_cast<const v4i*>(m + r * 128 + ((2 * lg + i) ^ (r & 7)) * 16);
      __builtin_memcpy(f + 4 * i, &x, 16);
    }
    split8<PARTS>(f, out);
  }
}

template <typename T, int PARTS, int C, bool WHOLE>
__global__ __launch_bounds__(4 * C, 4) void linear_gates_kernel(const LinGates a, long first, long units) {
  using Tile = GateTile<T, C, WHOLE>;
  constexpr int RT = C / 16, STEP = 128 / (int)sizeof(T);   // columns a step
  constexpr int MINE = kDotParts / RT;                      // parts of b and c a wave, at most
  __shared__ __attribute__((aligned(16))) unsigned char mq[Tile::BYTES], mk[Tile::BYTES], mo[Tile::BYTES], mv[Tile::BYTES];
  __shared__ double G[C];                       // inclusive sums of g, in powers of two
  __shared__ float pairs[RT][C];                // by strips of j, of each t
  __shared__ float sum_b[RT][C], sum_c[RT][C];  // by waves
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  // Blocks go round robin over the 8 XCDs; each takes neighbouring units, which are the heads of a chunk: rows
  // of one head lie a power of two apart and share few channels of an L2.
  const long per = (units + 7) / 8;
  for (long b = blockIdx.x; b < 8 * per; b += gridDim.x) {
    const long unit = b % 8 * per + b / 8;
    if (unit >= units) continue;
    const long item = first + unit / a.Hv;
    const int h = (int)(unit % a.Hv);
    LinItem it;
    if (!lin_item(a, item, &it) || it.len == 0) {
      if (threadIdx.x == 0 && a.ldg == 0) a.sums[item * a.Hv + h] = 0.f;
      continue;
    }
    const int n = it.len, hk = h / a.group;
    const long t0 = it.start;
    auto row = [&](const void* p, long ld, int head, int d) {
      return (const unsigned char*)p + (t0 * ld + (long)head * d) * (long)sizeof(T);
    };
    const unsigned char *qb = row(a.q, a.ldq, hk, a.dk), *kb = row(a.k, a.ldk, hk, a.dk);
    const unsigned char *ob = row(a.dout, a.lddout, h, a.dv), *vb = row(a.v, a.ldv, h, a.dv);
    Tile tq, tk, to, tv;
    auto fetch = [&](int s) {
      const int c0 = s * STEP;
      tq.fetch(qb, (unsigned)a.ldq, n, c0, a.dk);
      tk.fetch(kb, (unsigned)a.ldk, n, c0, a.dk);
      to.fetch(ob, (unsigned)a.lddout, n, c0, a.dv);
      tv.fetch(vb, (unsigned)a.ldv, n, c0, a.dv);
    };
    const float g = lane < n ? a.g[(t0 + lane) * a.ldg + h] : 0.f;
    float bs[MINE], cs[MINE];
    {
      const size_t at = (size_t)h * a.tokens + t0 + (lane < n ? lane : 0), step = (size_t)a.Hv * a.tokens;
#pragma unroll
      for (int i = 0; i < MINE; ++i) {
        const int part = w + RT * i < a.parts ? w + RT * i : 0;
        bs[i] = a.dots[at + part * step];
        cs[i] = a.dotk[at + part * step];
      }
    }
    fetch(0);
    if (w == 0) {
      double x = (g < -200.f ? -200.0 : (double)g) * 1.4426950408889634;   // as the passes have it
#pragma unroll
      for (int off = 1; off < C; off <<= 1) {
        const double y = __shfl_up(x, off);
        if (lane >= off) x += y;
      }
      if (lane < C) G[lane] = x;
    }
    {
      float sb = 0.f, sc = 0.f;
#pragma unroll
      for (int i = 0; i < MINE; ++i) {
        const bool in = w + RT * i < a.parts && lane < n;
        sb += in ? bs[i] : 0.f;
        sc += in ? cs[i] : 0.f;
      }
      if (lane < C) {
        sum_b[w][lane] = sb;
        sum_c[w][lane] = sc;
      }
    }
    v4f y[RT], z[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) y[i] = z[i] = v4f{0.f, 0.f, 0.f, 0.f};
    const int wide = a.dk > a.dv ? a.dk : a.dv;
    for (int s = 0; s * STEP < wide; ++s) {
      const int c0 = s * STEP;
      if (s > 0) __syncthreads();   // the tiles are free
      tq.stage(mq, c0, a.dk);
      tk.stage(mk, c0, a.dk);
      to.stage(mo, c0, a.dv);
      tv.stage(mv, c0, a.dv);
      __syncthreads();
      if (c0 + STEP < wide) fetch(s + 1);
      auto products = [&](const unsigned char* x, const unsigned char* m, v4f (&acc)[RT]) {
#pragma unroll
        for (int ks = 0; ks < STEP / 32; ++ks) {
          v8bf rows[PARTS];
          gate_operand<T, PARTS>(x, w, ks, rows);
#pragma unroll
          for (int i = 0; i < RT; ++i)
            if (i <= w) {
              v8bf cols[PARTS];
              gate_operand<T, PARTS>(m, i, ks, cols);
              acc[i] = mfma_parts<3>(rows, cols, acc[i]);
            }
        }
      };
      if (c0 < a.dk) products(mq, mk, y);
      if (c0 < a.dv) products(mo, mv, z);
    }
    // a lane has rows j = j0 + e and, of tile i, column 16 i + lr, which is the pairs' i and then t
    const int j0 = 16 * w + 4 * lg;
    double Gj[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) Gj[e] = G[j0 + e];
    float run[4] = {0.f, 0.f, 0.f, 0.f};   // the row's sums over the tiles so far
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int col = 16 * i + lr;
      float sum = 0.f;
      if (i <= w) {
        const double Gi = G[col];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = j0 + e;
          const bool low = j > col && j < n;
          float x = low ? y[i][e] * z[i][e] * (exp_diff(low ? Gj[e] - Gi : 0.0) * a.scale) : 0.f;
          x += dpp<0x111>(x);   // over the 16 lanes up to each: row_shr 1, 2, 4, 8
          x += dpp<0x112>(x);
          x += dpp<0x114>(x);
          x += dpp<0x118>(x);
          const float before = run[e] + dpp<0x111>(x);   // of the columns below t = col
          sum += j >= col ? before : 0.f;
          run[e] += dpp<0x15F>(x);                       // row_newbcast 15: the tile's
        }
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
      }
      if (lg == 0) pairs[w][col] = sum;
    }
    __syncthreads();
    if (w == 0) {   // t = lane
      const bool in = lane < n;
      float after = 0.f, up = 0.f, inside = 0.f;
      if (lane < C) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          after += sum_b[i][lane];
          up += sum_c[i][lane];
          inside += pairs[i][lane];
        }
      }
      const float whole = __shfl(up, n - 1);
      up = lane < n - 1 ? up : 0.f;
#pragma unroll
      for (int off = 1; off < C; off <<= 1) {
        const float s = __shfl_down(after, off), t = __shfl_up(up, off);
        if (lane + off < C) after += s;
        if (lane >= off) up += t;
      }
      up = __shfl_up(up, 1);
      const float dg = expf(g) == 0.f ? 0.f : inside + after + (lane > 0 ? up : 0.f) + whole;
      if (a.ldg) {
        if (in) a.dg[(t0 + lane) * a.Hv + h] = dg;
      } else {
        double total = in ? dg : 0.f;
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) total += __shfl_xor(total, off);
        if (lane == 0) a.sums[item * a.Hv + h] = (float)total;
      }
    }
    __syncthreads();   // LDS is free
  }
}

// dg of one decay a head: the chunks' sums, always in the same order.
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

template <typename T, int PARTS, int C>
hipError_t gates(const LinGates& a, long first, long units, hipStream_t s) {
  const long blocks = (units + 7) / 8 * 8;
  const unsigned grid = (unsigned)(blocks < (1L << 22) ? blocks : 1L << 22);   // threads are counted in 32 bits
  if (a.dk % 8 == 0 && a.dv % 8 == 0)
    linear_gates_kernel<T, PARTS, C, true><<<grid, 4 * C, 0, s>>>(a, first, units);
  else
    linear_gates_kernel<T, PARTS, C, false><<<grid, 4 * C, 0, s>>>(a, first, units);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_gates(const LinGates& a, hipStream_t s) {
  const bool all_long = !a.offsets && a.each > a.segment, all_short = !a.offsets && !all_long;
  const long first = all_long ? a.sequences : 0, last = all_short ? a.sequences : a.sequences + a.slots;
  const long units = (last - first) * a.Hv;
  hipError_t e = hipSuccess;
  if (units > 0)
    e = a.dtype == S4DPLR_BF16  ? gates<bf16, 1, 64>(a, first, units, s)
        : a.dtype == S4DPLR_F16 ? (a.segment == 64 ? gates<f16, 2, 64>(a, first, units, s)
                                                   : gates<f16, 2, 32>(a, first, units, s))
                                : (a.segment == 64 ? gates<float, 3, 64>(a, first, units, s)
                                                   : gates<float, 3, 32>(a, first, units, s));
  if (e != hipSuccess || a.ldg) return e;
  linear_gate_sums_kernel<<<dim3((unsigned)a.Hv), 256, 0, s>>>(a.sums, first, last, a.Hv, a.dg);
  return hipGetLastError();
}

}  // namespace s4
