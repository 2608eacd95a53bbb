// serve_i8.hip -- gfx950 kernels and C-ABI of 8-bit rows with one scale each
// and of their product (declared in serve/qrow_i8.h).

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "qr_internal.h"
#include "qrow.h"
#include "serve/qrow_i8.h"

namespace {

typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int WAVE = 64;
constexpr int ROW_ALIGN = 128;   // bytes: qr_i8_row_bytes

__device__ __forceinline__ float bf16_value(uint16_t h) { return __builtin_bit_cast(float, (uint32_t)h << 16); }

// fp32 to bf16, round to nearest even (NaN stays NaN).
__device__ __forceinline__ uint16_t bf16_bits(float f) {
  const uint32_t u = __builtin_bit_cast(uint32_t, f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return (uint16_t)((u >> 16) | 0x40u);
  return (uint16_t)((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}

// ---------------------------------------------------------------------------
// the row quantizer

constexpr int RQ_THREADS = 256;

// Eight values of a row from element `at` on; zeros behind n. `vec`: the row
// starts on a 16-byte border, so that whole groups of eight load as vectors.
template <int SRC>
__device__ __forceinline__ void load8(const void* row, int at, int n, bool vec, float (&v)[8]) {
  if (vec && at + 8 <= n) {
    if (SRC == QR_BF16) {
      const u16x8 h = *reinterpret_cast<const u16x8*>(reinterpret_cast<const uint16_t*>(row) + at);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = bf16_value(h[i]);
    } else {
      const f32x4* p = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(row) + at);
      const f32x4 a = p[0], b = p[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0.0f;
      if (at + i < n)
        v[i] = SRC == QR_BF16 ? bf16_value(reinterpret_cast<const uint16_t*>(row)[at + i])
                              : reinterpret_cast<const float*>(row)[at + i];
    }
  }
}

__device__ __forceinline__ u32x2 pack_codes(const float (&v)[8], float inv) {
  u32x2 o;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint32_t u = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) u |= ((uint32_t)(int)__builtin_rintf(v[4 * w + i] * inv) & 0xffu) << (8 * i);
    o[w] = u;
  }
  return o;
}

// One workgroup per row. A row of up to 256 * 8 * KEEP values stays in
// registers between its maximum and its codes; what is longer is read again.
// Bound by the row's load, its reduction and its store: one pass over memory.
template <int SRC, int KEEP>
__global__ __launch_bounds__(RQ_THREADS) void k_quantize_rows_i8(const void* __restrict__ x, int n, int64_t x_stride,
                                                                 int64_t row_bytes, int8_t* __restrict__ codes,
                                                                 float* __restrict__ scales) {
  __shared__ uint32_t wave_max[RQ_THREADS / WAVE];
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x;
  constexpr int ESIZE = SRC == QR_BF16 ? 2 : 4;
  const uint8_t* row = reinterpret_cast<const uint8_t*>(x) + r * x_stride * ESIZE;
  const bool vec = ((uintptr_t)row & 15) == 0;
  const int n_vec = (int)(row_bytes >> 3);
  float keep[KEEP][8];
  // magnitudes compare as integers, and a NaN or an infinity beats every
  // finite value there
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    load8<SRC>(row, (tid + k * RQ_THREADS) * 8, n, vec, keep[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t m = __builtin_bit_cast(uint32_t, keep[k][i]) & 0x7fffffffu;
      top = m > top ? m : top;
    }
  }
  for (int g = tid + KEEP * RQ_THREADS; g < n_vec; g += RQ_THREADS) {
    float v[8];
    load8<SRC>(row, g * 8, n, vec, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t m = __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu;
      top = m > top ? m : top;
    }
  }
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)top, s);
    top = o > top ? o : top;
  }
  if ((tid & (WAVE - 1)) == 0) wave_max[tid / WAVE] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < RQ_THREADS / WAVE; ++w) top = wave_max[w] > top ? wave_max[w] : top;
  const float amax = __builtin_bit_cast(float, top);
  const bool finite = top < 0x7f800000u;
  float inv = 127.0f / amax;
  float d = amax / 127.0f;
  if (!finite || !(inv < __builtin_inff())) {
    inv = 0.0f;
    d = finite ? 0.0f : __builtin_nanf("");
  }
  int8_t* out = codes + r * row_bytes;
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    const int g = tid + k * RQ_THREADS;
    if (g < n_vec) *reinterpret_cast<u32x2*>(out + (int64_t)g * 8) = finite ? pack_codes(keep[k], inv) : u32x2{0, 0};
  }
  for (int g = tid + KEEP * RQ_THREADS; g < n_vec; g += RQ_THREADS) {
    float v[8];
    load8<SRC>(row, g * 8, n, vec, v);
    *reinterpret_cast<u32x2*>(out + (int64_t)g * 8) = finite ? pack_codes(v, inv) : u32x2{0, 0};
  }
  if (tid == 0) scales[r] = d;
}

template <int SRC>
int launch_quantize(const void* x, int64_t n_rows, int n, int64_t x_stride, int64_t rb, int8_t* codes, float* scales,
                    hipStream_t s) {
  const dim3 grid((uint32_t)n_rows), block(RQ_THREADS);
  if (rb <= RQ_THREADS * 8)
    hipLaunchKernelGGL((k_quantize_rows_i8<SRC, 1>), grid, block, 0, s, x, n, x_stride, rb, codes, scales);
  else if (rb <= 2 * RQ_THREADS * 8)
    hipLaunchKernelGGL((k_quantize_rows_i8<SRC, 2>), grid, block, 0, s, x, n, x_stride, rb, codes, scales);
  else
    hipLaunchKernelGGL((k_quantize_rows_i8<SRC, 6>), grid, block, 0, s, x, n, x_stride, rb, codes, scales);
  return qr_check_launch("k_quantize_rows_i8");
}

// ---------------------------------------------------------------------------
// the product

struct Product {
  const int8_t* w;
  const int8_t* x;
  const float* wd;
  const float* xd;
  const float* bias;
  void* y;
  int64_t y_stride;
  int n_out, n_tok, row_bytes;
};

template <int DST>
__device__ __forceinline__ void store_one(void* y, int64_t at, float v) {
  if (DST == QR_BF16) reinterpret_cast<uint16_t*>(y)[at] = bf16_bits(v);
  else reinterpret_cast<float*>(y)[at] = v;
}

__device__ __forceinline__ float scaled(int sum, float xd, float wd, float bias) {
  return ((float)sum * xd) * wd + bias;
}

// 64 output channels x 64 tokens per workgroup, a 32 x 32 quarter per wave,
// 128 values of the sum per step through LDS. The weights are the matrix
// instruction's left operand: a lane then ends with four neighbouring
// channels of one token.
constexpr int T_OUT = 64, T_TOK = 64, T_K = 128;
constexpr int T_PITCH = T_K + 16;   // bytes of a staged row

template <int DST>
__global__ __launch_bounds__(256) void k_matmul_i8(Product p) {
  __shared__ __attribute__((aligned(16))) int8_t sw[T_OUT * T_PITCH];
  __shared__ __attribute__((aligned(16))) int8_t sx[T_TOK * T_PITCH];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int li = lane & 15, lk = lane >> 4;
  const int out_tiles = (p.n_out + T_OUT - 1) / T_OUT;
  const int o0 = (int)(blockIdx.x % out_tiles) * T_OUT, t0 = (int)(blockIdx.x / out_tiles) * T_TOK;
  const int wo = (wave & 1) * 32, wt = (wave >> 1) * 32;
  i32x4 acc[2][2] = {};
  for (int k0 = 0; k0 < p.row_bytes; k0 += T_K) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = (tid >> 3) + 32 * i, col = (tid & 7) * 16;
      // rows behind the last repeat it: their results are not stored
      const int wr = o0 + row < p.n_out ? o0 + row : p.n_out - 1;
      const int xr = t0 + row < p.n_tok ? t0 + row : p.n_tok - 1;
      const i32x4 a = *reinterpret_cast<const i32x4*>(p.w + (int64_t)wr * p.row_bytes + k0 + col);
      const i32x4 b = *reinterpret_cast<const i32x4*>(p.x + (int64_t)xr * p.row_bytes + k0 + col);
      *reinterpret_cast<i32x4*>(sw + row * T_PITCH + col) = a;
      *reinterpret_cast<i32x4*>(sx + row * T_PITCH + col) = b;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < T_K; kk += 64) {
      i32x4 a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i] = *reinterpret_cast<const i32x4*>(sw + (wo + 16 * i + li) * T_PITCH + kk + 16 * lk);
        b[i] = *reinterpret_cast<const i32x4*>(sx + (wt + 16 * i + li) * T_PITCH + kk + 16 * lk);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], b[j], acc[i][j], 0, 0, 0);
    }
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int tok = t0 + wt + 16 * j + li;
    if (tok >= p.n_tok) continue;
    const float xd = p.xd[tok];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int o = o0 + wo + 16 * i + 4 * lk + e;
        if (o < p.n_out)
          store_one<DST>(p.y, (int64_t)tok * p.y_stride + o, scaled(acc[i][j][e], xd, p.wd[o], p.bias ? p.bias[o] : 0.0f));
      }
  }
}

template <int DST>
int launch_product(const Product& p, hipStream_t s) {
  const int64_t tiles = (int64_t)((p.n_out + T_OUT - 1) / T_OUT) * ((p.n_tok + T_TOK - 1) / T_TOK);
  if (tiles > UINT32_MAX / 256) return qr_fail(QR_EOVERFLOW, "n_out and n_tok need too many tiles for one launch");
  hipLaunchKernelGGL((k_matmul_i8<DST>), dim3((uint32_t)tiles), dim3(256), 0, s, p);
  return qr_check_launch("k_matmul_i8");
}

}  // namespace

extern "C" {

size_t qr_i8_row_bytes(int64_t n_per_row) {
  if (n_per_row <= 0 || n_per_row > QR_I8_MAX_IN) return 0;
  return (size_t)((n_per_row + ROW_ALIGN - 1) / ROW_ALIGN * ROW_ALIGN);
}

int qr_quantize_rows_i8(int src, const void* x, int64_t n_rows, int64_t n_per_row, int64_t x_stride, int8_t* codes,
                        float* scales, void* stream) {
  qr_clear_error();
  if (src != QR_F32 && src != QR_BF16) return qr_fail(QR_EINVAL_TYPE, "source type %d is not QR_F32 or QR_BF16", src);
  const int64_t rb = (int64_t)qr_i8_row_bytes(n_per_row);
  if (rb == 0)
    return qr_fail(QR_EINVAL_SHAPE, "n_per_row=%lld must be in 1..%d", (long long)n_per_row, QR_I8_MAX_IN);
  if (n_rows < 0 || x_stride < n_per_row) return qr_fail(QR_EINVAL_SHAPE, "negative n_rows, or x_stride below n_per_row");
  if (n_rows == 0) return QR_OK;
  if (n_rows > UINT32_MAX / RQ_THREADS || x_stride > INT64_MAX / 4 / n_rows)
    return qr_fail(QR_EOVERFLOW, "n_rows=%lld is more than one launch holds", (long long)n_rows);
  if (!x || !codes || !scales) return qr_fail(QR_EINVAL_PTR, "x, codes and scales must be non-NULL");
  if (!qr_aligned(x, src == QR_BF16 ? 2 : 4) || !qr_aligned(codes, 16) || !qr_aligned(scales, 4))
    return qr_fail(QR_EINVAL_PTR, "codes must be 16-byte aligned, x and scales to their elements");
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return src == QR_BF16 ? launch_quantize<QR_BF16>(x, n_rows, (int)n_per_row, x_stride, rb, codes, scales, s)
                        : launch_quantize<QR_F32>(x, n_rows, (int)n_per_row, x_stride, rb, codes, scales, s);
}

int qr_matmul_i8(const int8_t* w, const float* wd, const int8_t* x, const float* xd, const float* bias, int64_t n_out,
                 int64_t n_tok, int64_t n_in, int dst, void* y, int64_t y_stride, void* stream) {
  qr_clear_error();
  if (dst != QR_F32 && dst != QR_BF16) return qr_fail(QR_EINVAL_TYPE, "output type %d is not QR_F32 or QR_BF16", dst);
  const int64_t rb = (int64_t)qr_i8_row_bytes(n_in);
  if (rb == 0) return qr_fail(QR_EINVAL_SHAPE, "n_in=%lld must be in 1..%d", (long long)n_in, QR_I8_MAX_IN);
  if (n_out < 0 || n_tok < 0 || y_stride < n_out)
    return qr_fail(QR_EINVAL_SHAPE, "negative n_out or n_tok, or y_stride below n_out");
  if (n_out == 0 || n_tok == 0) return QR_OK;
  if (n_out > INT32_MAX - 256 || n_tok > INT32_MAX - 256 || y_stride > INT64_MAX / 4 / n_tok)
    return qr_fail(QR_EOVERFLOW, "n_out or n_tok too large");
  if (!w || !wd || !x || !xd || !y) return qr_fail(QR_EINVAL_PTR, "w, wd, x, xd and y must be non-NULL");
  if (!qr_aligned(w, 16) || !qr_aligned(x, 16) || !qr_aligned(wd, 4) || !qr_aligned(xd, 4) || !qr_aligned(bias, 4) ||
      !qr_aligned(y, dst == QR_BF16 ? 2 : 4))
    return qr_fail(QR_EINVAL_PTR, "codes must be 16-byte aligned, wd, xd, bias and y to their elements");
  const Product p = {w, x, wd, xd, bias, y, y_stride, (int)n_out, (int)n_tok, (int)rb};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dst == QR_BF16 ? launch_product<QR_BF16>(p, s) : launch_product<QR_F32>(p, s);
}

}  // extern "C"
