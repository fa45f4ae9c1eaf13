// Linear attention, chunked: the pass over a segment and the sums of a segment, as templates
// that linear_bf16.hip, linear_f16.hip and linear_f32.hip instantiate for their type.
//
// Over a chunk of C tokens, with G the inclusive sums of g, e_i = exp G_i, d_j = exp(G_C - G_j):
//   P = lower(exp(G_i - G_j) X Y^T),  O = read e (X S) + pair P W,  S <- exp(G_C) S + update Y^T (d W).
// From the ends of the sequences (rev) the chunk's rows are taken in reverse, and G_i is the sum of g
// over the rows behind row i of the chunk's order, without its own: the same formulas.
//
// A block of four waves walks over a segment's chunks.  Wave w holds CW columns of the state in
// registers, in the matrix instruction's result layout, which is also its operand layout for X S
// once the rows of Y^T are permuted (delta_prep.hip).  X, Y, W lie in LDS as bf16 parts; P is shared out
// by strips of 16 rows and passed through LDS.  The next chunk's rows are on their way in
// registers.
#pragma once

#include "linear_device.h"

namespace s4 {

// Eight elements of a row on their way, `at` bytes behind `base` (uniform).  WHOLE: rows have a
// multiple of 8 elements.  Columns behind d come from the row's start and are not used.
template <typename T, bool WHOLE>
__device__ __forceinline__ void fetch8(const unsigned char* __restrict__ base, unsigned at, int col,
                                       int d, T (&t)[8]) {
  if constexpr (WHOLE) {
    __builtin_memcpy(t, base + (at + (col < d ? col : 0) * (unsigned)sizeof(T)), sizeof(t));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      __builtin_memcpy(&t[i], base + (at + (col + i < d ? col + i : 0) * (unsigned)sizeof(T)), sizeof(T));
  }
}

// A tile of C rows x COLS columns of a tensor's head, on its way to LDS.
template <typename T, int PARTS, int C, int COLS, bool WHOLE>
struct LinTile {
  static constexpr int LD = COLS + 8, N = C * COLS / 8 / 256, STEP = 256 / (COLS / 8);
  static_assert(N * 256 * 8 == C * COLS, "");
  T v[N][8];
  // `n` rows from `base` on, ld elements apart (64 rows of less than 2^24 elements: offsets of
  // 32 bits), in reverse with rev; columns c0 and on
  __device__ __forceinline__ void fetch(const unsigned char* base, unsigned ld, int n, int rev, int c0,
                                        int d) {
    const int r0 = threadIdx.x / (COLS / 8), c = c0 + threadIdx.x % (COLS / 8) * 8;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      int row = r0 + i * STEP;
      row = row < n ? row : n - 1;   // behind the end: a row that is there, unused
      row = rev ? n - 1 - row : row;
      fetch8<T, WHOLE>(base, (unsigned)row * (ld * (unsigned)sizeof(T)), c, d, v[i]);
    }
  }
  __device__ __forceinline__ void stage(__bf16 (*to)[C][LD], int n, int c0, int d) const {
    const int r0 = threadIdx.x / (COLS / 8), c = threadIdx.x % (COLS / 8) * 8;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = r0 + i * STEP;
      if constexpr (WHOLE && sizeof(T) == 2 && PARTS == 1) {
        v8bf x;
        __builtin_memcpy(&x, v[i], 16);
        typedef int v4i __attribute__((ext_vector_type(4)));
        v4i y;
        __builtin_memcpy(&y, v[i], 16);
        y = r < n && c0 + c < d ? y : v4i{0, 0, 0, 0};
        *reinterpret_cast<v4i*>(&to[0][r][c]) = y;
      } else {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          x[j] = r < n && c0 + c + (WHOLE ? 0 : j) < d ? to_f32(v[i][j]) : 0.f;
        v8bf parts[PARTS];
        split8<PARTS>(x, parts);
#pragma unroll
        for (int q = 0; q < PARTS; ++q) *reinterpret_cast<v8bf*>(&to[q][r][c]) = parts[q];
      }
    }
  }
};

// A head's state: row 4 g + e of tile t is row 32 (t / 2) + 8 g + 4 (t % 2) + e of dx, g = lane / 16.
template <int TILES, int CT>
__device__ __forceinline__ void store_state(float* __restrict__ to, int col0, int dx, int dw, int rs,
                                            int cs, const v4f (&S)[TILES][CT]) {
  const int lr = threadIdx.x & 15, lg = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    const int col = col0 + 16 * c + lr;
    if (col >= dw) continue;
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      const int row = 32 * (t >> 1) + 8 * lg + 4 * (t & 1);
      float* at = to + (row * rs + col * cs);
      if (row + 4 <= dx) {
        if (rs == 1) {
          __builtin_memcpy(at, &S[t][c], 16);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) at[e * rs] = S[t][c][e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (row + e < dx) at[e * rs] = S[t][c][e];
      }
    }
  }
}
// Read without a load under a condition: 0 where there is none.
template <int TILES, int CT>
__device__ __forceinline__ void load_state(const float* __restrict__ from, int col0, int dx, int dw,
                                           int rs, int cs, v4f (&S)[TILES][CT]) {
  const int lr = threadIdx.x & 15, lg = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int t = 0; t < TILES; ++t)
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int row = 32 * (t >> 1) + 8 * lg + 4 * (t & 1), col = col0 + 16 * c + lr;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool in = col < dw && row + e < dx;
        const float v = from[in ? (row + e) * rs + col * cs : 0];
        S[t][c][e] = in ? v : 0.f;
      }
    }
}

enum { kSum, kOut, kGrad };   // what a segment adds; a pass; a pass with `dot` and out in float

template <typename T, int PARTS, int DX, int CW, int C, bool WHOLE, int MODE>
__global__ __launch_bounds__(256, PARTS == 1 && DX <= 128 ? 2 : 1) void linear_pass_kernel(
    const LinPass p) {
  constexpr int TILES = DX / 16, CT = CW / 16, KS = DX / 32, RT = C / 16, COLS = 4 * CW;
  constexpr bool SUM = MODE == kSum;
  using XTile = LinTile<T, PARTS, C, DX, WHOLE>;
  using WTile = LinTile<T, PARTS, C, COLS, WHOLE>;
  __shared__ __attribute__((aligned(16))) __bf16 ys[PARTS][C][DX + 8];
  __shared__ __attribute__((aligned(16))) __bf16 ws[PARTS][C][COLS + 8];
  __shared__ __attribute__((aligned(16))) __bf16 xs[SUM ? 1 : PARTS][SUM ? 1 : C][DX + 8];
  __shared__ __attribute__((aligned(16))) __bf16 ps[SUM ? 1 : 3][SUM ? 1 : C][C + 8];
  __shared__ float2 G[C];
  __shared__ __attribute__((aligned(16))) float es[C], ds[C];
  __shared__ float whole;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lg = lane >> 4;
  const int slices = (p.dw + COLS - 1) / COLS;
  // blocks go round robin over the 8 XCDs; the slices of a head share one
  const unsigned g8 = blockIdx.x >> 3;
  const int slice = g8 % slices;
  const unsigned unit = g8 / slices * 8 + (blockIdx.x & 7);
  // items to be found: all sequences, or slots alone
  const long skip = p.offsets || p.each <= p.segment ? (SUM ? p.sequences : 0) : p.sequences;
  const int h = unit % p.Hv;
  LinItem it;
  if (!lin_item(p, skip + unit / p.Hv, &it)) return;
  if (it.of == 0 && it.len <= p.step_tokens) return;
  // the segment that is processed last has nobody to add to
  if (SUM && (p.rev ? it.m == 0 : it.m == it.of - 1)) return;
  const int len = it.len, chunks = (len + C - 1) / C;
  const int col0 = slice * COLS + w * CW;
  const size_t sz = (size_t)p.dk * p.dv;
  const int rs = (int)p.rs, cs = (int)p.cs;

  v4f S[TILES][CT];
#pragma unroll
  for (int t = 0; t < TILES; ++t)
#pragma unroll
    for (int c = 0; c < CT; ++c) S[t][c] = v4f{0.f, 0.f, 0.f, 0.f};
  if constexpr (!SUM) {
    const float* from = it.of ? p.before + ((size_t)it.slot * p.Hv + h) * sz
                              : p.first ? p.first + ((size_t)it.s * p.Hv + h) * sz : nullptr;
    if (from) load_state(from, col0, p.dx, p.dw, rs, cs, S);
    if (p.copy && !it.of)
      store_state(p.copy + ((size_t)it.s * p.Hv + h) * sz, col0, p.dx, p.dw, rs, cs, S);
  }

  XTile xr, yr;
  WTile wr;
  float gr = 0.f;
  double all = 0.0;   // the segment's decay
  // the head's columns in the segment's first row
  typedef const unsigned char* Bytes;
  const Bytes xb = (Bytes)p.x + (it.start * p.ldx + (long)(h / p.gx) * p.dx) * (long)sizeof(T);
  const Bytes yb = (Bytes)p.y + (it.start * p.ldy + (long)(h / p.gy) * p.dx) * (long)sizeof(T);
  const Bytes wb = (Bytes)p.w + (it.start * p.ldw + (long)(h / p.gw) * p.dw) * (long)sizeof(T);
  const float* gb = p.g ? p.g + it.start * p.ldg + h : nullptr;
  const long ldo = (long)p.Hv * p.dw;
  // first row and number of rows of chunk i of this pass's order
  auto first_of = [&](int i) { return (p.rev ? chunks - 1 - i : i) * C; };
  auto rows_of = [&](int c0) { return len - c0 < C ? len - c0 : C; };
  auto fetch = [&](int i) {
    const int c0 = first_of(i), n = rows_of(c0);
    if constexpr (!SUM)
      xr.fetch(xb + c0 * (p.ldx * (long)sizeof(T)), (unsigned)p.ldx, n, p.rev, 0, p.dx);
    yr.fetch(yb + c0 * (p.ldy * (long)sizeof(T)), (unsigned)p.ldy, n, p.rev, 0, p.dx);
    wr.fetch(wb + c0 * (p.ldw * (long)sizeof(T)), (unsigned)p.ldw, n, p.rev, slice * COLS, p.dw);
    if (w == 0 && gb) {
      const int row = lane < n ? p.rev ? n - 1 - lane : lane : 0;
      gr = gb[(c0 + row) * p.ldg];
      gr = lane < n ? gr : 0.f;
    }
  };
  if (chunks > 0) fetch(0);
  for (int i = 0; i < chunks; ++i) {
    const int c0 = first_of(i), n = rows_of(c0);
    if (w == 0) {
      // decays as powers of two, summed in 64 bits, so that a difference keeps its digits behind
      // a large negative g (a reset); below -200 the decay is 0 in fp32 either way
      const double own = (gr < -200.f ? -200.0 : (double)gr) * 1.4426950408889634;
      double x = own;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const double y = __shfl_up(x, off);
        if (lane >= off) x += y;
      }
      const double last = __shfl(x, 63);
      if (p.rev) x -= own;
      if (lane < C) {
        const float hi = (float)x;
        G[lane] = float2{hi, (float)(x - hi)};
        es[lane] = exp_diff(x) * p.read;
        ds[lane] = exp_diff(last - x) * p.update;
      }
      if (lane == 0) whole = exp_diff(last);
      all += last;
    }
    if constexpr (!SUM) xr.stage(xs, n, 0, p.dx);
    yr.stage(ys, n, 0, p.dx);
    wr.stage(ws, n, slice * COLS, p.dw);
    __syncthreads();
    if (i + 1 < chunks) fetch(i + 1);

    v4f O[SUM ? 1 : RT][CT];
    if constexpr (!SUM) {
      // P's rows 16 w .. + 16, a lane one row and four neighbouring columns of each tile
      if (w < RT) {
        v8bf xo[KS][PARTS];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int q = 0; q < PARTS; ++q)
            xo[ks][q] = *reinterpret_cast<const v8bf*>(&xs[q][16 * w + lr][32 * ks + 8 * lg]);
        const float2 gi = G[16 * w + lr];
#pragma unroll
        for (int ct = 0; ct < RT; ++ct) {
          if (ct > (w | 1)) continue;   // never read
          v4f acc = {0.f, 0.f, 0.f, 0.f};
          if (ct <= w) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              v8bf yo[PARTS];
#pragma unroll
              for (int q = 0; q < PARTS; ++q)
                yo[q] = *reinterpret_cast<const v8bf*>(&ys[q][16 * ct + lr][32 * ks + 8 * lg]);
              acc = mfma_parts<3>(yo, xo[ks], acc);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = 16 * ct + 4 * lg + e;
              const float2 gj = G[j];
              const float f = __builtin_amdgcn_exp2f((gi.x - gj.x) + (gi.y - gj.y));
              acc[e] = j <= 16 * w + lr ? acc[e] * f * p.pair : 0.f;
            }
          }
          v4bf parts[3];
          split4<3>(acc, parts);
#pragma unroll
          for (int q = 0; q < 3; ++q)
            *reinterpret_cast<v4bf*>(&ps[q][16 * w + lr][16 * ct + 4 * lg]) = parts[q];
        }
      }
      // X S, transposed: a lane one row and four neighbouring columns
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) O[r][c] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        v8bf so[CT][3];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          float t[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            t[e] = S[2 * ks][c][e];
            t[4 + e] = S[2 * ks + 1][c][e];
          }
          split8<3>(t, so[c]);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          v8bf xo[PARTS];
#pragma unroll
          for (int q = 0; q < PARTS; ++q)
            xo[q] = *reinterpret_cast<const v8bf*>(&xs[q][16 * r + lr][32 * ks + 8 * lg]);
#pragma unroll
          for (int c = 0; c < CT; ++c) O[r][c] = mfma_parts<3>(so[c], xo, O[r][c]);
        }
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float e = es[16 * r + lr];
#pragma unroll
        for (int c = 0; c < CT; ++c) O[r][c] *= e;
      }
    }
    {
      const float a = whole;
#pragma unroll
      for (int t = 0; t < TILES; ++t)
#pragma unroll
        for (int c = 0; c < CT; ++c) S[t][c] *= a;
    }
    if constexpr (!SUM) __syncthreads();   // P is there
#pragma unroll
    for (int ks = 0; ks < C / 32; ++ks) {
      v8bf wo[CT][PARTS];
#pragma unroll
      for (int c = 0; c < CT; ++c) get_tr<PARTS, 4>(ws, 32 * ks, w * CW + 16 * c, lr, lg, wo[c]);
      if constexpr (!SUM) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          if (ks > r / 2) continue;   // above the diagonal
          v8bf po[3];
#pragma unroll
          for (int q = 0; q < 3; ++q)
            po[q] = *reinterpret_cast<const v8bf*>(&ps[q][16 * r + lr][32 * ks + 8 * lg]);
#pragma unroll
          for (int c = 0; c < CT; ++c) O[r][c] = mfma_parts<3>(wo[c], po, O[r][c]);
        }
      }
      v8bf dw[CT][3];
      float d[8];
      __builtin_memcpy(d, &ds[32 * ks + 8 * lg], sizeof(d));
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        float t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float v = (float)wo[c][0][j];
#pragma unroll
          for (int q = 1; q < PARTS; ++q) v += (float)wo[c][q][j];
          t[j] = v * d[j];
        }
        split8<3>(t, dw[c]);
      }
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        v8bf yo[PARTS];
        get_tr<PARTS, 8>(ys, 32 * ks, 32 * (t >> 1) + 4 * (t & 1), lr, lg, yo);
#pragma unroll
        for (int c = 0; c < CT; ++c) S[t][c] = mfma_parts<3>(yo, dw[c], S[t][c]);
      }
    }
    if constexpr (!SUM) {
      // rows of out of this chunk: base (uniform) and offsets of 32 bits
      const long tok0 = it.start + c0;
      const unsigned wide = MODE == kGrad && p.out_f32 ? 4 : sizeof(T);
      unsigned char* ob = (unsigned char*)p.out + (tok0 * ldo + (long)h * p.dw) * wide;
      const Bytes db = MODE == kGrad
          ? (Bytes)p.dot + (tok0 * p.lddot + (long)(h / p.gdot) * p.dw) * (long)sizeof(T) : nullptr;
      float* to = MODE == kGrad && p.dot
          ? p.dot_out + ((size_t)(slice * 4 + w) * p.Hv + h) * p.tokens + tok0 : nullptr;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int i = 16 * r + lr, row = p.rev ? n - 1 - i : i;
        float sum = 0.f;
        if (i < n) {
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            const int col = col0 + 16 * c + 4 * lg;
            const v4f o = O[r][c];
            auto put = [&](int e0, int m) {   // columns e0 .. e0 + m of the four
              unsigned char* q = ob + ((unsigned)row * ((unsigned)ldo * wide) + (col + e0) * wide);
              if (MODE == kGrad && p.out_f32) {
                __builtin_memcpy(q, (const float*)&o + e0, 4 * m);
              } else if (MODE == kOut || p.out) {
                T t[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) t[e] = from_f32<T>(o[e]);
                __builtin_memcpy(q, t + e0, sizeof(T) * m);
              }
              if (MODE == kGrad && p.dot) {
                T t[4];
                __builtin_memcpy(t, db + ((unsigned)row * ((unsigned)p.lddot * (unsigned)sizeof(T)) +
                                          (col + e0) * (unsigned)sizeof(T)), sizeof(T) * m);
                for (int e = 0; e < m; ++e) sum = fmaf(o[e0 + e], to_f32(t[e]), sum);
              }
            };
            if (col + 4 <= p.dw) {
              put(0, 4);
            } else if constexpr (!WHOLE) {
              if (col < p.dw) put(0, 1);
              if (col + 1 < p.dw) put(1, 1);
              if (col + 2 < p.dw) put(2, 1);
            }
          }
        }
        if (MODE == kGrad && p.dot) {   // over the lanes that share the row
          sum += __shfl_xor(sum, 16);
          sum += __shfl_xor(sum, 32);
          if (lg == 0 && i < n) to[row] = sum;
        }
      }
    }
    __syncthreads();   // LDS is free
  }

  if constexpr (SUM) {
    store_state(p.states + ((size_t)it.slot * p.Hv + h) * sz, col0, p.dx, p.dw, rs, cs, S);
    if (threadIdx.x == 0 && slice == 0) p.decay[(size_t)it.slot * p.Hv + h] = exp_diff(all);
  } else {
    if (p.last && (it.of == 0 || (p.rev ? it.m == 0 : it.m == it.of - 1)))
      store_state(p.last + ((size_t)it.s * p.Hv + h) * sz, col0, p.dx, p.dw, rs, cs, S);
    if (MODE == kOut && p.edge_out) {
      const float* with = it.of ? p.edge_slots + ((size_t)it.slot * p.Hv + h) * sz
                                : p.edge_first + ((size_t)it.s * p.Hv + h) * sz;
      v4f other[TILES][CT];
      load_state(with, col0, p.dx, p.dw, rs, cs, other);
      float sum = 0.f;
#pragma unroll
      for (int t = 0; t < TILES; ++t)
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum = fmaf(S[t][c][e], other[t][c][e], sum);
      sum = sum64(sum);
      const size_t item = it.of ? (size_t)p.sequences + it.slot : (size_t)it.s;
      if (lane == 0) p.edge_out[(item * p.Hv + h) * kDotParts + slice * 4 + w] = sum;
    }
  }
}

// The variant for these sizes: f(DX, CW, C as constants).  The columns of the state that a wave
// holds: 32, or 16 where the head has no more than 64 or the operands' parts leave no room in
// LDS; chunks of 32 tokens where 64 do not fit.
template <int PARTS, typename F>
void linear_shape(int dx, int dw, F f) {
  using std::integral_constant;
#define S4_CASE(DX, CW, C) \
  f(integral_constant<int, DX>(), integral_constant<int, CW>(), integral_constant<int, C>())
  if (dx <= 64) {
    if (dw <= 64 || PARTS == 3) S4_CASE(64, 16, 64);
    else if constexpr (PARTS < 3) S4_CASE(64, 32, 64);
  } else if (dx <= 128) {
    if (dw <= 64 || PARTS > 1) S4_CASE(128, 16, 64);
    else if constexpr (PARTS == 1) S4_CASE(128, 32, 64);
  } else {
    if constexpr (PARTS == 1) S4_CASE(256, 16, 64);
    else S4_CASE(256, 16, 32);
  }
#undef S4_CASE
}

template <typename T, int PARTS, int MODE>
hipError_t linear_launch(const LinPass& a, hipStream_t s) {
  const bool all_long = !a.offsets && a.each > a.segment, all_short = !a.offsets && !all_long;
  const long items = (all_long || MODE == kSum ? 0 : a.sequences) + (all_short ? 0 : a.slots);
  if (items == 0) return hipSuccess;
  linear_shape<PARTS>(a.dx, a.dw, [&](auto dx, auto cw, auto c) {
    constexpr int DX = decltype(dx)::value, CW = decltype(cw)::value, C = decltype(c)::value;
    const long units = items * a.Hv;
    const unsigned grid = (unsigned)((units + 7) / 8 * 8 * ((a.dw + 4 * CW - 1) / (4 * CW)));
    if (a.dx % 8 == 0 && a.dw % 8 == 0)
      linear_pass_kernel<T, PARTS, DX, CW, C, true, MODE><<<grid, 256, 0, s>>>(a);
    else
      linear_pass_kernel<T, PARTS, DX, CW, C, false, MODE><<<grid, 256, 0, s>>>(a);
  });
  return hipGetLastError();
}

}  // namespace s4
