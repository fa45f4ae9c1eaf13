// Host side of the root-mean-square norm, quantization to 8 bits and the 8-bit product:
// argument validation.
#include <hip/hip_runtime_api.h>

#include <cmath>

#include "buffers.h"
#include "fp8.h"
#include "norm.h"
#include "rms.h"

namespace {

using namespace s4;

s4dplr_status rms_shape(long rows, long D) {
  if (rows < 0 || rows >= (1L << 31) || D < 1 || D > kNormMaxD) return S4DPLR_ERR_SHAPE;
  return S4DPLR_OK;
}

size_t rms_part_bytes(long rows, long D) {
  return align_up(sizeof(float) * (size_t)norm_parts(rows, D, 1) * (size_t)D);
}

size_t groups(long n) { return (size_t)(n + 127) / 128; }

// Bytes from the first to the last of `rows` rows of `width` bytes, `ld` apart.
size_t span(long rows, long ld, long width) {
  return rows > 0 && width > 0 ? (size_t)(rows - 1) * ld + width : 0;
}

constexpr long kMostSize = 1L << 24;   // rows, columns and pitches of an 8-bit operand

}  // namespace

extern "C" {

s4dplr_status s4dplr_rms_norm_fwd(const void* x, const void* residual, const float* gamma, void* h,
                                  void* y, void* q, void* scales, float* rstd, long rows, long D,
                                  float eps, int dtype, hipStream_t stream) {
  if (!valid_dtype(dtype)) return S4DPLR_ERR_UNSUPPORTED;
  if (s4dplr_status st = rms_shape(rows, D)) return st;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return S4DPLR_ERR_SHAPE;
  if (!q != !scales) return S4DPLR_ERR_NULL;
  if (rows == 0) return S4DPLR_OK;
  if (!x || (!y && !q)) return S4DPLR_ERR_NULL;
  const size_t es = elem(dtype), n = (size_t)rows * D;
  const Buf in[] = {{residual, n * es, es}, {x, n * es, es}, {gamma, sizeof(float) * (size_t)D, 4}};
  const Buf out[] = {{h, n * es, es},
                     {y, n * es, es},
                     {q, n, 1},
                     {scales, (size_t)rows * groups(D), 1},
                     {rstd, sizeof(float) * (size_t)rows, 4}};
  if (s4dplr_status st = check_buffers(in, out, 0, 0)) return st;
  RmsArgs a = {};
  a.x = x;
  a.residual = residual;
  a.gamma = gamma;
  a.h = h;
  a.y = y;
  a.q = static_cast<unsigned char*>(q);
  a.scales = static_cast<unsigned char*>(scales);
  a.rstd = rstd;
  a.rows = rows;
  a.D = D;
  a.eps = eps;
  return done(launch_rms_fwd(a, dtype, stream));
}

s4dplr_status s4dplr_rms_norm_workspace_bytes(long rows, long D, size_t* bytes) {
  if (!bytes) return S4DPLR_ERR_NULL;
  if (s4dplr_status st = rms_shape(rows, D)) return st;
  *bytes = rms_part_bytes(rows, D);
  return S4DPLR_OK;
}

s4dplr_status s4dplr_rms_norm_bwd(const void* h, const float* gamma, const float* rstd,
                                  const void* dy, const void* dh, void* dx, float* dgamma,
                                  long rows, long D, int dtype, void* ws, hipStream_t stream) {
  if (!valid_dtype(dtype)) return S4DPLR_ERR_UNSUPPORTED;
  if (s4dplr_status st = rms_shape(rows, D)) return st;
  if (rows > 0 && (!h || !rstd || !dy)) return S4DPLR_ERR_NULL;
  if (!ws) return S4DPLR_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(ws) % kAlign) return S4DPLR_ERR_WORKSPACE;
  const size_t es = elem(dtype), n = (size_t)rows * D, gb = sizeof(float) * (size_t)D;
  const Buf in[] = {{dh, n * es, es}, {h, n * es, es}, {gamma, gb, 4},
                    {rstd, sizeof(float) * (size_t)rows, 4}, {dy, n * es, es}};
  const Buf out[] = {{dx, n * es, es}, {dgamma, gb, 4}, {ws, rms_part_bytes(rows, D), kAlign}};
  if (s4dplr_status st = check_buffers(in, out, 0, 0)) return st;
  if (!dgamma && (!dx || rows == 0)) return S4DPLR_OK;
  RmsArgs a = {};
  a.x = h;
  a.gamma = gamma;
  a.rstd = const_cast<float*>(rstd);
  a.dy = dy;
  a.dh = dh;
  a.dx = dx;
  a.dgamma = dgamma;
  a.part = static_cast<float*>(ws);
  a.rows = rows;
  a.D = D;
  return done(launch_rms_bwd(a, dtype, stream));
}

s4dplr_status s4dplr_quantize_fp8(const void* x, long ldx, void* q, void* scales, void* qt,
                                  void* scales_t, long rows, long cols, int square, int dtype,
                                  hipStream_t stream) {
  if (!valid_dtype(dtype)) return S4DPLR_ERR_UNSUPPORTED;
  if (rows < 0 || cols < 0 || rows > kMostSize / 4 || cols >= kMostSize || ldx < cols ||
      ldx >= kMostSize)
    return S4DPLR_ERR_SHAPE;
  // a launch counts its threads, 512 a block, in 32 bits
  if (groups(rows) * groups(cols) >= (1u << 22)) return S4DPLR_ERR_SHAPE;
  if (!q != !scales || !qt != !scales_t) return S4DPLR_ERR_NULL;
  if (rows == 0 || cols == 0 || (!q && !qt)) return S4DPLR_OK;
  if (!x) return S4DPLR_ERR_NULL;
  const size_t es = elem(dtype), n = (size_t)rows * cols;
  const size_t down = square ? groups(rows) : (size_t)rows, across = square ? groups(cols) : (size_t)cols;
  const Buf in[] = {{x, es * span(rows, ldx, cols), es}};
  const Buf out[] = {{q, n, 1}, {scales, down * groups(cols), 1},
                     {qt, n, 1}, {scales_t, across * groups(rows), 1}};
  if (s4dplr_status st = check_buffers(in, out, -1, -1)) return st;
  QuantizeArgs a = {};
  a.x = x;
  a.ldx = ldx;
  a.q = static_cast<unsigned char*>(q);
  a.scales = static_cast<unsigned char*>(scales);
  a.qt = static_cast<unsigned char*>(qt);
  a.scales_t = static_cast<unsigned char*>(scales_t);
  a.rows = (int)rows;
  a.cols = (int)cols;
  a.square = square != 0;
  return done(launch_quantize(a, dtype, stream));
}

s4dplr_status s4dplr_matmul_fp8(const void* a, long lda, const void* a_scales, const void* b,
                                long ldb, const void* b_scales, int b_square, void* out, long ldo,
                                long M, long N, long K, int dtype, hipStream_t stream) {
  if (!valid_dtype(dtype)) return S4DPLR_ERR_UNSUPPORTED;
  for (long n : {M, N, K})
    if (n < 0 || n >= kMostSize) return S4DPLR_ERR_SHAPE;
  if (lda < K || ldb < K || ldo < N || lda >= kMostSize || ldb >= kMostSize || ldo >= kMostSize)
    return S4DPLR_ERR_SHAPE;
  // a launch counts its threads in 32 bits: tiles of 128 x 128 have 256 threads each and are no more than these,
  // smaller and larger ones are fewer (matmul.hip)
  if (((size_t)M + 63) / 64 * groups(N) >= (1u << 23)) return S4DPLR_ERR_SHAPE;
  if (M == 0 || N == 0) return S4DPLR_OK;
  if (!out || (K > 0 && (!a || !a_scales || !b || !b_scales))) return S4DPLR_ERR_NULL;
  const size_t es = elem(dtype);
  const Buf in[] = {{a, span(M, lda, K), 1}, {a_scales, (size_t)M * groups(K), 1},
                    {b, span(N, ldb, K), 1},
                    {b_scales, (b_square ? groups(N) : (size_t)N) * groups(K), 1}};
  const Buf res[] = {{out, es * span(M, ldo, N), es}};
  if (s4dplr_status st = check_buffers(in, res, -1, -1)) return st;
  MatmulArgs m = {};
  m.a = static_cast<const unsigned char*>(a);
  m.sa = static_cast<const unsigned char*>(a_scales);
  m.b = static_cast<const unsigned char*>(b);
  m.sb = static_cast<const unsigned char*>(b_scales);
  m.lda = lda;
  m.ldb = ldb;
  m.ldo = ldo;
  m.out = out;
  m.M = (int)M;
  m.N = (int)N;
  m.K = (int)K;
  m.square = b_square != 0;
  return done(launch_matmul(m, dtype, stream));
}

}  // extern "C"
