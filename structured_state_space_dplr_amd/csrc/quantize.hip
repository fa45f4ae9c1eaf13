// Quantization of a matrix x [rows][cols] to e4m3 with a power of two as the scale of each 128
// values: by rows (q, the operand of a product over the columns), by columns (qt, the
// transposed matrix, the operand of a product over the rows), or by 128 x 128 blocks (weights,
// for which one rounding serves both).  One pass over x writes both.
//
// A block takes a tile of 128 x 128.  A lane holds 16 bytes of each of neighbouring rows, so
// that a row's group lies in neighbouring lanes, and a column's values that one lane holds
// are 4 (16-bit) or 8 (fp32) neighbouring bytes of the transposed tile, which goes through LDS.
// Bound by HBM where there are tiles for every CU (8192 x 4096 of bf16, both forms: 33 us, 4.1 TB/s),
// by a tile's own loads, barriers and stores below (1003 x 1040 of fp16 5.5 us).
#include "fp8.h"
#include "fp8_device.h"
#include "vec.h"

namespace s4 {

namespace {
constexpr int kThreads = 512;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const QuantizeArgs a) {
  constexpr int VEC = Vec<T>::N;          // columns a lane
  constexpr int LANES = kGroup / VEC;     // lanes a row
  constexpr int SETS = kThreads / LANES;      // sets of neighbouring rows
  constexpr int R = kGroup / SETS;        // rows a set
  __shared__ unsigned red[SETS][kGroup];
  __shared__ unsigned all[kThreads / 64];
  // byte (c, r) of the transposed tile at 128 c + R (set ^ (c / VEC)) + r % R, so that the lanes of a
  // write lie apart
  __shared__ __attribute__((aligned(16))) unsigned char turned[kGroup * kGroup];
  const int tid = threadIdx.x, lane = tid % LANES, set = tid / LANES;
  const int r0 = blockIdx.y * kGroup, c0 = blockIdx.x * kGroup;
  const int col = c0 + lane * VEC, row = r0 + set * R;
  const int cg = (a.cols + kGroup - 1) / kGroup, rg = (a.rows + kGroup - 1) / kGroup;
  const T* x = (const T*)a.x;
  const bool rows = a.q && blockIdx.z == 0, columns = a.qt && blockIdx.z == gridDim.z - 1;
  float v[R][VEC];
  if (r0 + kGroup <= a.rows && c0 + kGroup <= a.cols) {
    Vec<T> t[R];
#pragma unroll
    for (int i = 0; i < R; ++i) t[i] = load_vec(x + (long)(row + i) * a.ldx + col);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = to_f32(t[i].v[j]);
  } else if (a.cols % VEC == 0) {
    // at the edge: every load from inside, all on their way together, and zeros behind the ends
    typedef int v4i __attribute__((ext_vector_type(4)));
    v4i t[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
      __builtin_memcpy(&t[i], x + (long)(row + i < a.rows ? row + i : a.rows - 1) * a.ldx + (col < a.cols ? col : 0), 16);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      asm volatile("" : "+v"(t[i]));   // or the loads are put under the condition, one by one, or split
      T u[VEC];
      __builtin_memcpy(u, &t[i], 16);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = row + i < a.rows && col < a.cols ? to_f32(u[j]) : 0.f;
    }
  } else {
    T t[R][VEC];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const T* p = x + (long)(row + i < a.rows ? row + i : a.rows - 1) * a.ldx;
#pragma unroll
      for (int j = 0; j < VEC; ++j) t[i][j] = p[col + j < a.cols ? col + j : 0];
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float f = to_f32(t[i][j]);
        asm volatile("" : "+v"(f));
        v[i][j] = row + i < a.rows && col + j < a.cols ? f : 0.f;
      }
  }
  unsigned block = 0;   // scale of the whole tile
  if (a.square) {
    unsigned big = 0;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const unsigned m = magnitude(v[i][j]);
        big = m > big ? m : big;
      }
    big = max_of<32>(big);
    const unsigned other = (unsigned)__shfl_xor((int)big, 32);
    big = other > big ? other : big;
    if (tid % 64 == 0) all[tid / 64] = big;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) big = all[i] > big ? all[i] : big;
    block = scale_byte(big);
    if (tid == 0) {
      if (rows) a.scales[(long)blockIdx.y * cg + blockIdx.x] = (unsigned char)block;
      if (columns) a.scales_t[(long)blockIdx.x * rg + blockIdx.y] = (unsigned char)block;
    }
  }
  if (rows) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      unsigned byte = block;
      if (!a.square) {
        unsigned big = 0;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const unsigned m = magnitude(v[i][j]);
          big = m > big ? m : big;
        }
        byte = scale_byte(max_of<LANES>(big));
      }
      const float f = inverse_scale(byte);
      unsigned t[VEC / 4];
#pragma unroll
      for (int j = 0; j < VEC; j += 4)
        t[j / 4] = pack4(v[i][j] * f, v[i][j + 1] * f, v[i][j + 2] * f, v[i][j + 3] * f);
      if (row + i >= a.rows) continue;   // behind the lanes' exchange
      unsigned char* p = a.q + (long)(row + i) * a.cols + col;
      if (col + VEC <= a.cols) {
        __builtin_memcpy(p, t, VEC);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (col + j < a.cols) p[j] = (unsigned char)(t[j / 4] >> (8 * (j % 4)));
      }
      if (!a.square && lane == 0) a.scales[(long)(row + i) * cg + blockIdx.x] = (unsigned char)byte;
    }
  }
  if (!columns) return;
  if (!a.square) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      unsigned big = 0;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const unsigned m = magnitude(v[i][j]);
        big = m > big ? m : big;
      }
      red[set][lane * VEC + j] = big;
    }
    __syncthreads();
    if (tid < kGroup) {
      unsigned big = 0;
#pragma unroll
      for (int i = 0; i < SETS; ++i) big = red[i][tid] > big ? red[i][tid] : big;
      const unsigned byte = scale_byte(big);
      red[0][tid] = byte;   // read and written by this thread alone before the barrier
      if (c0 + tid < a.cols) a.scales_t[(long)(c0 + tid) * rg + blockIdx.y] = (unsigned char)byte;
    }
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const float f = inverse_scale(a.square ? block : red[0][lane * VEC + j]);
    unsigned t[R / 4];
#pragma unroll
    for (int i = 0; i < R; i += 4)
      t[i / 4] = pack4(v[i][j] * f, v[i + 1][j] * f, v[i + 2][j] * f, v[i + 3][j] * f);
    __builtin_memcpy(&turned[(lane * VEC + j) * kGroup + R * (set ^ (lane % SETS))], t, R);
  }
  __syncthreads();
  constexpr int STEP = kThreads / SETS;   // columns a pass
  const int s = tid % SETS;
#pragma unroll
  for (int i = 0; i < kGroup / STEP; ++i) {
    const int c = i * STEP + tid / SETS;
    if (c0 + c >= a.cols) break;
    unsigned char t[R];
    __builtin_memcpy(t, &turned[c * kGroup + R * (s ^ (c / VEC % SETS))], R);
    const int r = r0 + s * R;
    unsigned char* p = a.qt + (long)(c0 + c) * a.rows + r;
    if (r + R <= a.rows) {
      __builtin_memcpy(p, t, R);
    } else {
#pragma unroll
      for (int k = 0; k < R; ++k)
        if (r + k < a.rows) p[k] = t[k];
    }
  }
}

hipError_t launch_quantize(const QuantizeArgs& a, int dtype, hipStream_t s) {
  const unsigned across = (a.cols + kGroup - 1) / kGroup, down = (a.rows + kGroup - 1) / kGroup;
  // Both forms of a tile by blocks of their own while there is a tile a CU at most: each is a chain of
  // steps that the other need not wait for (fp16, us): 1024 x 2048 4.6 against 5.4, 2048 x 2048 6.1 and
  // 6.2; fp32 7.4 and 8.1; above, the tile's second read costs more: fp32 2048 x 4096 13.1 and 11.8.
  const unsigned apart = a.q && a.qt && (long)across * down <= 256 ? 2 : 1;
  const dim3 grid(across, down, apart);
  if (dtype == S4DPLR_F32) quantize_kernel<float><<<grid, kThreads, 0, s>>>(a);
  else if (dtype == S4DPLR_BF16) quantize_kernel<bf16><<<grid, kThreads, 0, s>>>(a);
  else quantize_kernel<f16><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace s4
