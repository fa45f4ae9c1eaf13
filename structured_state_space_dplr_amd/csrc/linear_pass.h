// Linear attention, chunked: the pass over a segment and the sums of a segment, as templates
// that linear_bf16.hip, linear_f16.hip and linear_f32.hip instantiate for their type.
//
// Over a chunk of C tokens, with G the inclusive sums of g, e_i = exp G_i, d_j = exp(G_C - G_j):
//   P = lower(exp(G_i - G_j) X Y^T),  O = read e (X S) + pair P W,  S <- exp(G_C) S + update Y^T (d W).
// From the ends of the sequences (rev) the chunk's rows are taken in reverse, and G_i is the sum of g
// over the rows behind row i of the chunk's order, without its own: the same formulas.
//
// A block of eight waves (four where the head has 64 columns or less, or the parts leave no room)
// walks over a segment's chunks.  Wave w holds CW columns of the state in
// registers, in the matrix instruction's result layout, which is also its operand layout for X S
// once the rows of Y^T are permuted (delta_prep.hip).  X, Y, W lie in LDS as bf16 parts; P is shared out
// by strips of 16 rows and passed through LDS.  The next chunk's rows are on their way in
// registers.
//
// What bounds it is the issue of instructions: in 16-bit 128 x 128 heads the vector units are busy 64 % of
// the CUs' time (splitting states and weights into parts, the decays, staging) and the matrix units
// 35 %, one after the other in a wave, with four waves a SIMD; LDS is at 46 %.  Eight waves a
// block, which share X, Y and P, against four: 160 us instead of 172 for a prompt of 16384 tokens of
// 16 heads.  Kernel times there (bf16): sums 36 us, states 15, pass 88; training step of 4 x 4096
// tokens: sums 44, states 14, passes 107 (o, dv) and, with what the decays' gradient needs of them, 159
// (dq; 235 MB of states written) and 171 (dk; the same read).
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

// Rows of tiles in LDS: their pieces of 16 bytes change places by the row's low bits.  Neither 16
// rows of one piece (an operand by rows) nor 4 rows of 4 neighbouring pieces (a transposing read)
// share banks then, for rows of 128 bytes or a multiple of 256.  Where a byte of a row lies is
// (byte ^ turn(row)); turn(row + 16) = turn(row), turn(row + 4) = turn(row) ^ 16 if row % 8 < 4.
template <int COLS>
__device__ __forceinline__ unsigned turn(unsigned row) {
  return COLS == 64 ? (row >> 1 & 1) << 6 | (row >> 2 & 3) << 4 : (row & 3) << 6 | (row >> 2 & 3) << 4;
}

typedef __attribute__((address_space(3))) unsigned char Lds;

__device__ __forceinline__ v8bf take(const Lds* at) {
  return *reinterpret_cast<const __attribute__((address_space(3))) v8bf*>(at);
}
// Operand of 16 columns by 32 rows: as get_tr (delta_device.h); `lo` are rows r .. r + 4 of a lane's
// share, `hi` the next four.
__device__ __forceinline__ v8bf take_tr(const Lds* lo, const Lds* hi) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) v4s lds4;
  union {
    v4s h[2];
    v8bf v;
  } u;
  u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)lo);
  u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)hi);
  return u.v;
}
template <typename V>
__device__ __forceinline__ void put(Lds* at, V v) {
  *reinterpret_cast<__attribute__((address_space(3))) V*>(at) = v;
}
template <typename V>
__device__ __forceinline__ V get(const Lds* at) {
  return *reinterpret_cast<const __attribute__((address_space(3))) V*>(at);
}

// c[i] += a b over the parts, for N independent c, which lie between two instructions of one.
template <int KEEP, int PA, int PB, typename F>
__device__ __forceinline__ void over_parts(F f) {
#pragma unroll
  for (int i = PA - 1; i >= 0; --i)
#pragma unroll
    for (int j = PB - 1; j >= 0; --j)
      if (i + j < KEEP) f(i, j);
}

// A tile of C rows x COLS columns of a tensor's head, on its way to LDS.
template <typename T, int PARTS, int C, int COLS, bool WHOLE, int THREADS>
struct LinTile {
  static constexpr int N = C * COLS / 8 / THREADS, STEP = THREADS / (COLS / 8);
  static constexpr int ROW = 2 * COLS, PART = C * ROW;   // bytes in LDS
  static_assert(N * THREADS * 8 == C * COLS && STEP % 8 == 0, "");
  T v[N][8];
  // `n` rows from `base` on, ld elements apart (64 rows of less than 2^24 elements: offsets of
  // 32 bits), in reverse with rev; columns c0 and on
  __device__ __forceinline__ void fetch(const unsigned char* base, unsigned ld, int n, int rev, int c0,
                                        int d) {
    const unsigned tid = thread(), r0 = tid / (COLS / 8);
    const int c = c0 + (int)(tid % (COLS / 8) * 8);
    const unsigned pitch = ld * (unsigned)sizeof(T);
    if (n == C) {
      const unsigned first = (rev ? C - 1 - r0 : r0) * pitch, step = rev ? 0u - STEP * pitch : STEP * pitch;
#pragma unroll
      for (int i = 0; i < N; ++i) fetch8<T, WHOLE>(base, first + i * step, c, d, v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        int row = (int)r0 + i * STEP;
        row = row < n ? row : n - 1;   // behind the end: a row that is there, unused
        row = rev ? n - 1 - row : row;
        fetch8<T, WHOLE>(base, (unsigned)row * pitch, c, d, v[i]);
      }
    }
  }
  __device__ __forceinline__ void stage(Lds* to, int n, int c0, int d) const {
    const unsigned tid = thread(), r0 = tid / (COLS / 8);
    const int c = (int)(tid % (COLS / 8) * 8);
    // rows 16 apart have one turn
    Lds* const first = to + (r0 * ROW | (2u * c ^ turn<COLS>(r0)));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = (int)r0 + i * STEP;
      Lds* at = STEP % 16 == 0 ? first + i * STEP * ROW : to + ((unsigned)(r * ROW) | (2u * c ^ turn<COLS>(r)));
      if constexpr (WHOLE && sizeof(T) == 2 && PARTS == 1) {
        typedef int v4i __attribute__((ext_vector_type(4)));
        v4i y;
        __builtin_memcpy(&y, v[i], 16);
        if (n < C || c0 + COLS > d) {
          asm volatile("");   // a branch: most tiles are whole
          y = r < n && c0 + c < d ? y : v4i{0, 0, 0, 0};
        }
        put(at, y);
      } else {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          x[j] = r < n && c0 + c + (WHOLE ? 0 : j) < d ? to_f32(v[i][j]) : 0.f;
        v8bf parts[PARTS];
        split8<PARTS>(x, parts);
#pragma unroll
        for (int q = 0; q < PARTS; ++q) put(at + q * PART, parts[q]);
      }
    }
  }
};

// A head's state: row 4 g + e of tile t is row 32 (t / 2) + 8 g + 4 (t % 2) + e of dx, g = lane / 16.
template <int TILES, int CT>
__device__ __forceinline__ void store_state(float* __restrict__ to, int col0, int dx, int dw, int rs,
                                            int cs, const v4f (&S)[TILES][CT]) {
  const unsigned tid = thread();
  const int lr = tid & 15, lg = (tid & 63) >> 4;
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
template <int TILES, int CT>
__device__ __forceinline__ void load_state(const float* __restrict__ from, int col0, int dx, int dw,
                                           int rs, int cs, v4f (&S)[TILES][CT], int first = 0) {
  const unsigned tid = thread();
  const int lr = tid & 15, lg = (tid & 63) >> 4;
  auto row_of = [&](int t) { return 32 * ((first + t) >> 1) + 8 * lg + 4 * ((first + t) & 1); };
  if (rs == 1 && dx % 4 == 0) {
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const int row = row_of(t), col = col0 + 16 * c + lr;
        __builtin_memcpy(&S[t][c], from + (col < dw && row < dx ? row + col * cs : 0), 16);
      }
  } else {
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = row_of(t) + e, col = col0 + 16 * c + lr;
          S[t][c][e] = from[col < dw && row < dx ? row * rs + col * cs : 0];
        }
  }
#pragma unroll
  for (int t = 0; t < TILES; ++t)
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v = S[t][c][e];
        touch(v);
        S[t][c][e] = col0 + 16 * c + lr < dw && row_of(t) + e < dx ? v : 0.f;
      }
}

enum { kSum, kOut, kGrad };   // what a segment adds; a pass; a pass with `dot` and out in float

// Blocks that share a CU: two where they fit into its LDS.
constexpr int linear_blocks(int parts, int dx, int cols, int c, int mode) {
  const int tiles = 2 * parts * c * (mode == kSum ? dx + cols : 2 * dx + cols);
  const int pairs = mode == kSum ? 0 : 6 * c * (c + 8);
  return 2 * (tiles + pairs + 2048) <= 160 * 1024 ? 2 : 1;
}

template <typename T, int PARTS, int DX, int WAVES, int CW, int C, bool WHOLE, int MODE>
__global__ __launch_bounds__(64 * WAVES, WAVES / 4 * linear_blocks(PARTS, DX, WAVES * CW, C, MODE))
void linear_pass_kernel(const LinPass p) {
  constexpr int TILES = DX / 16, CT = CW / 16, KS = DX / 32, RT = C / 16, COLS = WAVES * CW;
  constexpr bool SUM = MODE == kSum;
  using XTile = LinTile<T, PARTS, C, DX, WHOLE, 64 * WAVES>;
  using WTile = LinTile<T, PARTS, C, COLS, WHOLE, 64 * WAVES>;
  // LDS: Y, W, (X, P by parts of C rows,) and of two chunks in turn G as pairs of floats, d, the whole decay
  constexpr int PROW = 2 * (C + 8), PPART = C * PROW;
  constexpr int oY = 0, oW = oY + PARTS * XTile::PART, oX = oW + PARTS * WTile::PART;
  constexpr int oP = oX + (SUM ? 0 : PARTS * XTile::PART), oG = oP + (SUM ? 0 : 3 * PPART);
  constexpr int oD = oG + 2 * 8 * C, oWhole = oD + 2 * 4 * C;
  __shared__ __attribute__((aligned(512))) unsigned char memory[oWhole + 8];
  Lds* const lds = (Lds*)memory;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
  // (the sums' pass goes the other way, so that a chunk's decay to the segment's end is known)
  auto first_of = [&](int i) { return ((p.rev != 0) != SUM ? chunks - 1 - i : i) * C; };
  auto rows_of = [&](int c0) { return len - c0 < C ? len - c0 : C; };
  auto fetch = [&](int i) {
    const int c0 = first_of(i), n = rows_of(c0);
    if constexpr (!SUM)
      xr.fetch(xb + c0 * (p.ldx * (long)sizeof(T)), (unsigned)p.ldx, n, p.rev, 0, p.dx);
    yr.fetch(yb + c0 * (p.ldy * (long)sizeof(T)), (unsigned)p.ldy, n, p.rev, 0, p.dx);
    wr.fetch(wb + c0 * (p.ldw * (long)sizeof(T)), (unsigned)p.ldw, n, p.rev, slice * COLS, p.dw);
  };
  // wave 0: g of chunk i, a row a lane, two chunks ahead of its use
  auto fetch_g = [&](int i) {
    if (w != 0 || !gb || i >= chunks) return;
    const int c0 = first_of(i), n = rows_of(c0), row = lane < n ? lane : n - 1;
    gr = gb[(c0 + (p.rev ? n - 1 - row : row)) * p.ldg];
  };
  // wave 0: the decays of chunk i as powers of two, summed in 64 bits, so that a difference keeps its
  // digits behind a large negative g (a reset); below -200 the decay is 0 in fp32 either way
  auto decays = [&](int i) {
    if (w != 0 || i >= chunks) return;
    const float g = lane < rows_of(first_of(i)) ? gr : 0.f;
    const double own = (g < -200.f ? -200.0 : (double)g) * 1.4426950408889634;
    double x = own;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const double y = __shfl_up(x, off);
      if (lane >= off) x += y;
    }
    const double last = __shfl(x, 63);
    if (p.rev) x -= own;
    // the sums' pass: `all` is the decay behind the chunk so far
    const double far = SUM ? last + all : last;
    if (lane < C) {
      const float hi = (float)x;
      put(lds + oG + ((i & 1) * 8 * C + 8 * lane), v2f{hi, (float)(x - hi)});
      put(lds + oD + ((i & 1) * 4 * C + 4 * lane), exp_diff(far - x) * p.update);
    }
    if (!SUM && lane == 0) put(lds + oWhole + (i & 1) * 4, exp_diff(last));
    all += last;
  };
  if (chunks > 0) {
    fetch_g(0);
    fetch(0);
    decays(0);
    fetch_g(1);
  }
  for (int i = 0; i < chunks; ++i) {
    const int c0 = first_of(i), n = rows_of(c0), at = i & 1;
    if constexpr (!SUM) xr.stage(lds + oX, n, 0, p.dx);
    yr.stage(lds + oY, n, 0, p.dx);
    wr.stage(lds + oW, n, slice * COLS, p.dw);
    __syncthreads();
    const long tok0 = it.start + c0;
    // the decays' gradient: row 0 of this wave's part of dot_out's rows of this chunk
    float* const part = MODE == kGrad && p.dot
        ? p.dot_out + ((size_t)(slice * WAVES + w) * p.Hv + h) * p.tokens + tok0 : nullptr;
    if (MODE == kGrad && p.dot) {
      // a wave's part of a state, as its lanes hold it
      constexpr size_t PART = TILES * CT * 64 * 4;
      float* const inner = p.inner + (((size_t)(tok0 / C) * p.Hv + h) * slices * WAVES + slice * WAVES + w) * PART
          + 4 * (thread() & 63);
      if (!p.rev) {
        if (c0 > 0)
#pragma unroll
          for (int t = 0; t < TILES; ++t)
#pragma unroll
            for (int c = 0; c < CT; ++c) __builtin_memcpy(inner + (t * CT + c) * 256, &S[t][c], 16);
      } else {
        // the inner product of the states on either side of the chunk, four tiles at a time; nothing where
        // the decay over the chunk is 0
        float across = 0.f;
        const float whole = get<float>(lds + oWhole + 4 * at);
        if (__builtin_amdgcn_readfirstlane(__float_as_uint(whole)) != 0) {
          const float* const from = it.of ? p.inner_slots + ((size_t)it.slot * p.Hv + h) * sz
                                          : p.inner_first + ((size_t)it.s * p.Hv + h) * sz;
#pragma unroll
          for (int t0 = 0; t0 < TILES; t0 += 4) {
            v4f other[4][CT];
            if (c0 > 0) {
#pragma unroll
              for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int c = 0; c < CT; ++c) __builtin_memcpy(&other[t][c], inner + ((t0 + t) * CT + c) * 256, 16);
            } else {
              load_state(from, col0, p.dx, p.dw, rs, cs, other, t0);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
              for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) across = fmaf(S[t0 + t][c][e], other[t][c][e], across);
            touch(across);
          }
          across = sum64(across) * whole;
        }
        if (lane == 0) part[n - 1] = across;
      }
    }
    if (i + 1 < chunks) fetch(i + 1);
    decays(i + 1);
    fetch_g(i + 2);

    v4f O[SUM ? 1 : RT][CT];
    if constexpr (!SUM) {
      // P by strips of 16 rows, whose tiles the waves share out; a lane has one row and four
      // neighbouring columns of a tile
      constexpr int SHARE = WAVES / RT;
      const int strip = w % RT;
      {
        const unsigned tid = thread(), r = tid & 15, g = (tid & 63) >> 4;
        const unsigned row = r * XTile::ROW | (16 * g ^ turn<DX>(r));
        v8bf xo[KS][PARTS];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int q = 0; q < PARTS; ++q)
            xo[ks][q] = take(lds + oX + q * XTile::PART + ((row ^ 64 * ks) + strip * 16 * XTile::ROW));
        const v2f gi = get<v2f>(lds + oG + (at * 8 * C + 8 * (16 * strip + r)));
#pragma unroll
        for (int k = 0; k < (RT + SHARE - 1) / SHARE; ++k) {
          const int ct = k * SHARE + w / RT;
          if (ct > (strip | 1)) continue;   // never read
          v4f acc = {0.f, 0.f, 0.f, 0.f};
          if (ct <= strip) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              v8bf yo[PARTS];
#pragma unroll
              for (int q = 0; q < PARTS; ++q)
                yo[q] = take(lds + oY + q * XTile::PART + ((row ^ 64 * ks) + ct * 16 * XTile::ROW));
              acc = mfma_parts<3>(yo, xo[ks], acc);
            }
            const Lds* gp = lds + oG + (at * 8 * C + 8 * (16 * ct + 4 * g));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const v2f gj = get<v2f>(gp + 8 * e);
              const float f = __builtin_amdgcn_exp2f((gi[0] - gj[0]) + (gi[1] - gj[1]));
              acc[e] = 16 * ct + 4 * g + e <= 16 * strip + r ? acc[e] * f * p.pair : 0.f;
            }
          }
          v4bf parts[3];
          split4<3>(acc, parts);
#pragma unroll
          for (int q = 0; q < 3; ++q)
            put(lds + oP + q * PPART + ((16 * strip + r) * PROW + 2 * (16 * ct + 4 * g)), parts[q]);
        }
      }
      // X S, transposed: a lane one row and four neighbouring columns
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) O[r][c] = v4f{0.f, 0.f, 0.f, 0.f};
      {
        const unsigned tid = thread(), lr = tid & 15, g = (tid & 63) >> 4;
        const unsigned row = lr * XTile::ROW | (16 * g ^ turn<DX>(lr));
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
          v8bf xo[RT][PARTS];
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int q = 0; q < PARTS; ++q)
              xo[r][q] = take(lds + oX + q * XTile::PART + r * 16 * XTile::ROW + (row ^ 64 * ks));
          over_parts<3, 3, PARTS>([&](int i, int j) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
              for (int c = 0; c < CT; ++c) O[r][c] = mfma(so[c][i], xo[r][j], O[r][c]);
          });
        }
        // (the zeros: or the registers of an array that is filled under a condition live through the whole
        // loop, and are spilled)
        T dot[MODE == kGrad ? RT : 1][CT][4] = {};
        if (MODE == kGrad && p.dot) {
          const unsigned tid = thread();
          const int lr = tid & 15, lg = (tid & 63) >> 4;
          const Bytes db = (Bytes)p.dot + (tok0 * p.lddot + (long)(h / p.gdot) * p.dw) * (long)sizeof(T);
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const int i = 16 * r + lr < n ? 16 * r + lr : n - 1;
            const unsigned at = (unsigned)(p.rev ? n - 1 - i : i) * ((unsigned)p.lddot * (unsigned)sizeof(T));
#pragma unroll
            for (int c = 0; c < CT; ++c) {
              const int col = col0 + 16 * c + 4 * lg;
              if constexpr (WHOLE) {
                __builtin_memcpy(dot[r][c], db + (at + (col < p.dw ? col : 0) * (unsigned)sizeof(T)), sizeof(dot[r][c]));
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  __builtin_memcpy(&dot[r][c][e], db + (at + (col + e < p.dw ? col + e : 0) * (unsigned)sizeof(T)),
                                   sizeof(T));
              }
            }
          }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const v2f gi = get<v2f>(lds + oG + (at * 8 * C + 8 * lr) + 8 * 16 * r);
          const float e = __builtin_amdgcn_exp2f(gi[0] + gi[1]) * p.read;
#pragma unroll
          for (int c = 0; c < CT; ++c) O[r][c] *= e;
          if (MODE == kGrad && p.dot) {   // columns behind dw: O is 0
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
              for (int e = 0; e < 4; ++e) sum = fmaf(O[r][c][e], to_f32(dot[r][c][e]), sum);
            // over the lanes that share the row
            const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(sum), __float_as_uint(sum), false, false);
            sum = __uint_as_float(a[0]) + __uint_as_float(a[1]);
            const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(sum), __float_as_uint(sum), false, false);
            sum = __uint_as_float(b[0]) + __uint_as_float(b[1]);
            const int i = 16 * r + lr;
            if (g == 0 && i < n && !(p.rev && i == 0)) part[p.rev ? n - 1 - i : i] = sum;
          }
        }
      }
    }
    if constexpr (!SUM) {
      const float a = get<float>(lds + oWhole + 4 * at);
#pragma unroll
      for (int t = 0; t < TILES; ++t)
#pragma unroll
        for (int c = 0; c < CT; ++c) S[t][c] *= a;
    }
    if constexpr (!SUM) __syncthreads();   // P is there
    {
      const unsigned tid = thread(), lr = tid & 15, g = (tid & 63) >> 4, row = 8 * g + (lr >> 2);
      // four rows of four groups of four columns: of W neighbouring ones, of Y 8 columns apart
      const unsigned wt = row * WTile::ROW | ((2 * CW * w + 8 * (lr & 3)) ^ turn<COLS>(row));
      const unsigned yt = row * XTile::ROW | (16 * (lr & 3) ^ turn<DX>(row));
#pragma unroll
      for (int ks = 0; ks < C / 32; ++ks) {
        v8bf wo[CT][PARTS];
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
          for (int q = 0; q < PARTS; ++q) {
            const Lds* m = lds + oW + q * WTile::PART + ks * 32 * WTile::ROW;
            wo[c][q] = take_tr(m + (wt ^ 32 * c), m + 4 * WTile::ROW + (wt ^ 32 * c ^ 16));
          }
        if constexpr (!SUM) {
#pragma unroll
          for (int r = 2 * ks; r < RT; r += 2) {   // two strips; those above are above the diagonal
            v8bf po[2][3];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int q = 0; q < 3; ++q)
                po[k][q] = take(lds + oP + q * PPART + 16 * (r + k) * PROW + 64 * ks + (lr * PROW + 16 * g));
            over_parts<3, PARTS, 3>([&](int i, int j) {
#pragma unroll
              for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int c = 0; c < CT; ++c) O[r + k][c] = mfma(wo[c][i], po[k][j], O[r + k][c]);
            });
          }
        }
        v8bf dw[CT][3];
        {
          const v4f d0 = get<v4f>(lds + oD + 128 * ks + (4 * C * at + 32 * g));
          const v4f d1 = get<v4f>(lds + oD + 128 * ks + 16 + (4 * C * at + 32 * g));
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            float t[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float v = (float)wo[c][0][j];
#pragma unroll
              for (int q = 1; q < PARTS; ++q) v += (float)wo[c][q][j];
              t[j] = v * (j < 4 ? d0[j & 3] : d1[j & 3]);
            }
            split8<3>(t, dw[c]);
          }
        }
#pragma unroll
        for (int t = 0; t < TILES; t += 4) {
          v8bf yo[4][PARTS];
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int q = 0; q < PARTS; ++q) {
              const Lds* m = lds + oY + q * XTile::PART + ks * 32 * XTile::ROW + 8 * (k & 1);
              const unsigned x = 64 * ((t + k) >> 1);
              yo[k][q] = take_tr(m + (yt ^ x), m + 4 * XTile::ROW + (yt ^ x ^ 16));
            }
          over_parts<3, PARTS, 3>([&](int i, int j) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int c = 0; c < CT; ++c) S[t + k][c] = mfma(yo[k][i], dw[c][j], S[t + k][c]);
          });
        }
      }
    }
    if constexpr (!SUM) {
      const unsigned tid = thread();
        const int lr = tid & 15, lg = (tid & 63) >> 4;
      // rows of out of this chunk: base (uniform) and offsets of 32 bits
      const unsigned wide = MODE == kGrad && p.out_f32 ? 4 : sizeof(T);
      unsigned char* ob = (unsigned char*)p.out + (tok0 * ldo + (long)h * p.dw) * wide;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int i = 16 * r + lr, row = p.rev ? n - 1 - i : i;
        if (i < n) {
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            const int col = col0 + 16 * c + 4 * lg;
            const v4f o = O[r][c];
            auto write = [&](int e0, int m) {   // columns e0 .. e0 + m of the four
              unsigned char* q = ob + ((unsigned)row * ((unsigned)ldo * wide) + (col + e0) * wide);
              if (MODE == kGrad && p.out_f32) {
                __builtin_memcpy(q, (const float*)&o + e0, 4 * m);
              } else if (p.out) {
                T t[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) t[e] = from_f32<T>(o[e]);
                __builtin_memcpy(q, t + e0, sizeof(T) * m);
              }
            };
            if (col + 4 <= p.dw) {
              write(0, 4);
            } else if constexpr (!WHOLE) {
              if (col < p.dw) write(0, 1);
              if (col + 1 < p.dw) write(1, 1);
              if (col + 2 < p.dw) write(2, 1);
            }
          }
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
  }
}

// The variant for these sizes: f(DX, WAVES, CW, C as constants).  A wave holds 16 columns of the
// state; eight share a block where the head has more than 64, unless the operands' parts leave no
// room in LDS.  Chunks of 32 tokens where 64 do not fit.
template <int PARTS, typename F>
void linear_shape(int dx, int dw, F f) {
  using std::integral_constant;
  constexpr integral_constant<int, 4> four;
  constexpr integral_constant<int, 8> eight;
  constexpr integral_constant<int, 16> cw;
  constexpr integral_constant<int, 64> c64;
  constexpr integral_constant<int, linear_chunk(256, PARTS)> c256;
  const bool wide = dw > 64;
  if (dx <= 64) {
    constexpr integral_constant<int, 64> d;
    if (wide) f(d, eight, cw, c64);
    else f(d, four, cw, c64);
  } else if (dx <= 128) {
    constexpr integral_constant<int, 128> d;
    if constexpr (PARTS < 3) {
      if (wide) return f(d, eight, cw, c64);
    }
    f(d, four, cw, c64);
  } else {
    constexpr integral_constant<int, 256> d;
    if (wide) f(d, eight, cw, c256);
    else f(d, four, cw, c256);
  }
}

template <typename T, int PARTS, int MODE>
hipError_t linear_launch(const LinPass& a, hipStream_t s) {
  const bool all_long = !a.offsets && a.each > a.segment, all_short = !a.offsets && !all_long;
  const long items = (all_long || MODE == kSum ? 0 : a.sequences) + (all_short ? 0 : a.slots);
  if (items == 0) return hipSuccess;
  linear_shape<PARTS>(a.dx, a.dw, [&](auto dx, auto waves, auto cw, auto c) {
    constexpr int DX = decltype(dx)::value, W = decltype(waves)::value, CW = decltype(cw)::value;
    constexpr int C = decltype(c)::value;
    const long units = items * a.Hv;
    const unsigned grid = (unsigned)((units + 7) / 8 * 8 * ((a.dw + W * CW - 1) / (W * CW)));
    if (a.dx % 8 == 0 && a.dw % 8 == 0)
      linear_pass_kernel<T, PARTS, DX, W, CW, C, true, MODE><<<grid, 64 * W, 0, s>>>(a);
    else
      linear_pass_kernel<T, PARTS, DX, W, CW, C, false, MODE><<<grid, 64 * W, 0, s>>>(a);
  });
  return hipGetLastError();
}

}  // namespace s4
