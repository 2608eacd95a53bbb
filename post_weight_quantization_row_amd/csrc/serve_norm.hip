// serve_norm.hip -- gfx950 kernel and C-ABI of the norm that makes 8-bit rows
// (declared in serve/qrow_norm.h).

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "qr_internal.h"
#include "qrow.h"
#include "serve/qrow_norm.h"
#include "serve_internal.h"

namespace {

using namespace serve;

struct Norm {
  const void* x;
  const void* residual;
  const void* weight;
  void* sum;
  void* y;
  int8_t* codes;
  float* scales;
  int64_t x_stride, residual_stride, sum_stride, y_stride, row_bytes;
  double eps;
  int n, n_rows, wtype;
};

template <int DST>
__device__ __forceinline__ void store8(void* row, int at, int n, const float (&v)[8]) {
  if (DST == QR_BF16) {
    uint16_t* p = reinterpret_cast<uint16_t*>(row) + at;
    if (at + 8 <= n) {
      u16x8_any h;
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = bf16_bits(v[i]);
      *reinterpret_cast<u16x8_any*>(p) = h;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (at + i < n) p[i] = bf16_bits(v[i]);
    }
  } else {
    float* p = reinterpret_cast<float*>(row) + at;
    if (at + 8 <= n) {
      *reinterpret_cast<f32x4_any*>(p) = f32x4_any{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4_any*>(p + 4) = f32x4_any{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (at + i < n) p[i] = v[i];
    }
  }
}

// Eight weights from element `at` on; zeros behind n, ones where there are none.
__device__ __forceinline__ void load_weights(const Norm& p, int at, float (&w)[8]) {
  if (!p.weight) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.0f;
  } else if (p.wtype == QR_BF16) {
    load8<QR_BF16>(p.weight, at, p.n, w);
  } else {
    load8<QR_F32>(p.weight, at, p.n, w);
  }
}

// The row's values from element `at` on: x plus the residual, rounded to the
// row's type, which the sum receives (the lane that reads an element is the one
// that writes it: in place is safe).
template <int SRC>
__device__ __forceinline__ void load_sum(const void* x, const void* residual, void* sum, int at, int n,
                                         float (&v)[8]) {
  load8<SRC>(x, at, n, v);
  if (!residual) return;
  float r[8];
  load8<SRC>(residual, at, n, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] += r[i];
    if (SRC == QR_BF16) v[i] = bf16_value(bf16_bits(v[i]));
  }
  store8<SRC>(sum, at, n, v);
}

// y = s * f, in fp32 after one rounding from 64 bits, times the weight. The
// row's factor stays in 64 bits: in 32 it would be subnormal, or zero, for rows
// of 1e38 and more.
__device__ __forceinline__ void normed(double f, const float (&w)[8], float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (float)((double)v[i] * f) * w[i];
}

__device__ __forceinline__ uint32_t largest(uint32_t top, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t m = __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu;
    top = m > top ? m : top;
  }
  return top;
}

// WAVES waves to a row. A row of up to 512 * WAVES * KEEP values stays in
// registers from its sum to its codes; what is longer is read again, twice. With
// eight waves and more, which are for few rows, the weights are asked for
// together with the row; else after its sum (16 registers less: a fifth wave per
// SIMD, though 12 values of a bf16 row lie in scratch memory then, 14 with KEEP 4;
// fp32 rows fit).
//
// Bound by one pass over memory: 8192 x 4096 bf16 with a residual 52 us, 4.5 TB/s
// (a copy passes at 4.6); one row 3.5 us, the time of its dependent steps. The
// 64-bit arithmetic costs nothing there (fp32 throughout: no faster). 8192 x 7168
// 135 us, 3.0 TB/s: four waves a SIMD, and more bytes than the Infinity Cache holds
// (8192 x 4096 out of it, the same rows again and again: 40 us).
template <int SRC, int WAVES, int KEEP>
__global__ __launch_bounds__(WAVES > 4 ? WAVES * WAVE : 256) __attribute__((amdgpu_waves_per_eu(KEEP == 2 && WAVES == 4 ? 5 : 4))) void k_norm_rows_i8(Norm p) {
  constexpr int LANES = WAVES * WAVE, ROWS = WAVES > 4 ? 1 : 4 / WAVES;
  constexpr bool AHEAD = KEEP == 1 || WAVES > 4;
  __shared__ double part[WAVES > 4 ? WAVES : 4];
  __shared__ uint32_t wave_max[WAVES > 4 ? WAVES : 4];
  constexpr int ESIZE = SRC == QR_BF16 ? 2 : 4;
  const int tid = threadIdx.x % LANES, wave = threadIdx.x / WAVE;
  const int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / LANES;
  if (WAVES == 1 && r >= p.n_rows) return;   // a wave by itself: nobody waits for it
  const uint8_t* x = reinterpret_cast<const uint8_t*>(p.x) + r * p.x_stride * ESIZE;
  const uint8_t* residual = p.residual ? reinterpret_cast<const uint8_t*>(p.residual) + r * p.residual_stride * ESIZE : nullptr;
  uint8_t* sum = p.residual ? reinterpret_cast<uint8_t*>(p.sum) + r * p.sum_stride * ESIZE : nullptr;
  uint8_t* y = p.y ? reinterpret_cast<uint8_t*>(p.y) + r * p.y_stride * ESIZE : nullptr;
  const uint8_t* again = sum ? sum : x;      // what a long row is read from later
  const int n_vec = (int)(p.row_bytes >> 3);
  float keep[KEEP][8], w[KEEP][8];
  double squares = 0.0;
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    load_sum<SRC>(x, residual, sum, (tid + k * LANES) * 8, p.n, keep[k]);
    if (AHEAD) load_weights(p, (tid + k * LANES) * 8, w[k]);
  }
#pragma unroll
  for (int k = 0; k < KEEP; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) squares = __builtin_fma((double)keep[k][i], (double)keep[k][i], squares);
  for (int g = tid + KEEP * LANES; g < n_vec; g += LANES) {
    float v[8];
    load_sum<SRC>(x, residual, sum, g * 8, p.n, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) squares = __builtin_fma((double)v[i], (double)v[i], squares);
  }
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) squares += __shfl_xor(squares, s);
  if (WAVES > 1) {
    if ((tid & (WAVE - 1)) == 0) part[wave] = squares;
    __syncthreads();
    squares = 0.0;
#pragma unroll
    for (int v = 0; v < WAVES; ++v) squares += part[v];
  }
  const double f = 1.0 / __builtin_sqrt(squares / (double)p.n + p.eps);
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    if (!AHEAD) load_weights(p, (tid + k * LANES) * 8, w[k]);
    normed(f, w[k], keep[k]);
    if ((tid + k * LANES) * 8 < p.n) {
      top = largest(top, keep[k]);
      if (y) store8<SRC>(y, (tid + k * LANES) * 8, p.n, keep[k]);
    }
  }
  for (int g = tid + KEEP * LANES; g < n_vec; g += LANES) {
    float v[8];
    load8<SRC>(again, g * 8, p.n, v);
    load_weights(p, g * 8, w[0]);
    normed(f, w[0], v);
    top = largest(top, v);
  }
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)top, s);
    top = o > top ? o : top;
  }
  if (WAVES > 1) {
    if ((tid & (WAVE - 1)) == 0) wave_max[wave] = top;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < WAVES; ++v) top = wave_max[v] > top ? wave_max[v] : top;
  }
  const CodeScale c = code_scale(top);
  int8_t* out = p.codes + r * p.row_bytes;
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    const int g = tid + k * LANES;
    if (g < n_vec) *reinterpret_cast<u32x2*>(out + (int64_t)g * 8) = c.finite ? pack_codes(keep[k], c.inv) : u32x2{0, 0};
  }
  for (int g = tid + KEEP * LANES; g < n_vec; g += LANES) {
    float v[8];
    load8<SRC>(again, g * 8, p.n, v);
    load_weights(p, g * 8, w[0]);
    normed(f, w[0], v);
    if (y) store8<SRC>(y, g * 8, p.n, v);
    *reinterpret_cast<u32x2*>(out + (int64_t)g * 8) = c.finite ? pack_codes(v, c.inv) : u32x2{0, 0};
  }
  if (tid == 0) p.scales[r] = c.d;
}

template <int SRC, int WAVES, int KEEP>
int launch(const Norm& p, hipStream_t s) {
  const uint32_t rows = WAVES > 4 ? 1 : 4 / WAVES, threads = WAVES > 4 ? WAVES * WAVE : 256;
  const uint32_t groups = ((uint32_t)p.n_rows + rows - 1) / rows;
  if (groups > UINT32_MAX / threads) return qr_fail(QR_EOVERFLOW, "n_rows=%d is more than one launch holds", p.n_rows);
  hipLaunchKernelGGL((k_norm_rows_i8<SRC, WAVES, KEEP>), dim3(groups), dim3(threads), 0, s, p);
  return qr_check_launch("k_norm_rows_i8");
}

template <int SRC>
int launch_norm(const Norm& p, hipStream_t s) {
  // Few rows: as many waves to each as it has pieces of 512, which is the least
  // time that one takes; many: half of them, which wait for each other less.
  // Measured, us: 1 x 4096 bf16 eight waves 3.6, four 4.1; 8192 x 4096 four
  // 52, eight 73; 333 x 7168 fp32 eight 11.4, four 11.9
  const bool few = p.n_rows <= 512;
  if (p.n <= 512) return launch<SRC, 1, 1>(p, s);
  if (p.n <= 2048) return launch<SRC, 4, 1>(p, s);
  if (p.n <= 4096) return few ? launch<SRC, 8, 1>(p, s) : launch<SRC, 4, 2>(p, s);
  if (p.n <= 8192) return few ? launch<SRC, 8, 2>(p, s) : launch<SRC, 4, 4>(p, s);
  return launch<SRC, 16, 2>(p, s);
}

struct Rows {
  const char* name;
  const void* p;
  int64_t stride;   // elements; bytes once it is known to be no more than that holds
};

}  // namespace

extern "C" int qr_norm_rows_i8(int src, const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                               int wtype, const void* weight, double eps, int64_t n_rows, int64_t n, void* sum,
                               int64_t sum_stride, void* y, int64_t y_stride, int8_t* codes, float* scales,
                               void* stream) {
  qr_clear_error();
  if (src != QR_F32 && src != QR_BF16) return qr_fail(QR_EINVAL_TYPE, "source type %d is not QR_F32 or QR_BF16", src);
  if (wtype != QR_F32 && wtype != QR_BF16) return qr_fail(QR_EINVAL_TYPE, "weight type %d is not QR_F32 or QR_BF16", wtype);
  const int64_t rb = (int64_t)qr_i8_row_bytes(n);
  if (rb == 0) return qr_fail(QR_EINVAL_SHAPE, "n=%lld must be in 1..%d", (long long)n, QR_I8_MAX_IN);
  if (!(eps >= 0.0) || !(eps < __builtin_inf())) return qr_fail(QR_EINVAL_SHAPE, "eps must be finite and not negative");
  if (n_rows < 0) return qr_fail(QR_EINVAL_SHAPE, "negative n_rows");
  if (!residual != !sum && n_rows > 0) return qr_fail(QR_EINVAL_PTR, "residual and sum must both be given or both be NULL");
  const int64_t esize = src == QR_BF16 ? 2 : 4;
  // inputs, then the outputs that may be one of them
  Rows rows[4] = {{"x", x, x_stride}, {"residual", residual, residual_stride}, {"sum", sum, sum_stride}, {"y", y, y_stride}};
  for (int i = 0; i < 4; ++i) {
    if (i > 0 && !rows[i].p) continue;
    if (rows[i].stride < n) return qr_fail(QR_EINVAL_SHAPE, "%s_stride=%lld is below n", rows[i].name, (long long)rows[i].stride);
  }
  if (n_rows == 0) return QR_OK;
  for (Rows& r : rows) {
    if (!r.p) continue;
    if (r.stride > INT64_MAX / 4 / n_rows) return qr_fail(QR_EOVERFLOW, "%s_stride is too large", r.name);
    r.stride *= esize;
  }
  if (n_rows > UINT32_MAX / 256) return qr_fail(QR_EOVERFLOW, "n_rows=%lld is more than one launch holds", (long long)n_rows);
  if (!x || !codes || !scales) return qr_fail(QR_EINVAL_PTR, "x, codes and scales must be non-NULL");
  for (int i = 0; i < 4; ++i)
    if (!qr_aligned(rows[i].p, (uintptr_t)esize)) return qr_fail(QR_EINVAL_PTR, "%s must be aligned to its elements", rows[i].name);
  if (!qr_aligned(weight, wtype == QR_BF16 ? 2 : 4) || !qr_aligned(codes, 16) || !qr_aligned(scales, 4))
    return qr_fail(QR_EINVAL_PTR, "codes must be 16-byte aligned, weight and scales to their elements");
  const int64_t row = n * esize, wbytes = weight ? n * (wtype == QR_BF16 ? 2 : 4) : 0;
  for (int o = 2; o < 4; ++o) {
    const Rows& a = rows[o];
    if (!a.p) continue;
    for (int i = 0; i < o; ++i) {
      const Rows& b = rows[i];
      if (!b.p || (i < 2 && a.p == b.p && (n_rows == 1 || a.stride == b.stride))) continue;
      if (rows_meet(a.p, a.stride, b.p, b.stride, row, n_rows))
        return qr_fail(QR_EINVAL_PTR, "%s and %s must not overlap", a.name, b.name);
    }
    if (rows_meet_range(a.p, a.stride, row, n_rows, weight, wbytes))
      return qr_fail(QR_EINVAL_PTR, "%s and weight must not overlap", a.name);
  }
  const int64_t cbytes = n_rows * rb, sbytes = n_rows * 4;
  for (int i = 0; i < 4; ++i)
    if (rows[i].p && (rows_meet_range(rows[i].p, rows[i].stride, row, n_rows, codes, cbytes) ||
                      rows_meet_range(rows[i].p, rows[i].stride, row, n_rows, scales, sbytes)))
      return qr_fail(QR_EINVAL_PTR, "codes and scales must not overlap %s", rows[i].name);
  if (rows_meet_range(codes, cbytes, cbytes, 1, scales, sbytes) || rows_meet_range(codes, cbytes, cbytes, 1, weight, wbytes) ||
      rows_meet_range(scales, sbytes, sbytes, 1, weight, wbytes))
    return qr_fail(QR_EINVAL_PTR, "codes, scales and weight must not overlap");
  const Norm p = {x, residual, weight, sum, y, codes, scales, x_stride, residual_stride, sum_stride, y_stride, rb, eps,
                  (int)n, (int)n_rows, wtype};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return src == QR_BF16 ? launch_norm<QR_BF16>(p, s) : launch_norm<QR_F32>(p, s);
}
