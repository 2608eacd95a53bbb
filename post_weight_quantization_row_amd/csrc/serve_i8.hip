// serve_i8.hip -- gfx950 kernels and C-ABI of 8-bit rows with one scale each
// and of their product (declared in serve/qrow_i8.h).

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "qr_internal.h"
#include "qrow.h"
#include "serve/qrow_i8.h"

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// Vectors at any element of the caller's rows, whose strides are free: memory
// instructions take them unaligned.
typedef uint16_t u16x8_any __attribute__((ext_vector_type(8), aligned(2)));
typedef uint16_t u16x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

constexpr int WAVE = 64;
constexpr int ROW_ALIGN = 128;   // bytes: qr_i8_row_bytes

__device__ __forceinline__ float bf16_value(uint16_t h) { return __builtin_bit_cast(float, (uint32_t)h << 16); }

// fp32 to bf16, round to nearest even (NaN stays NaN).
__device__ __forceinline__ uint16_t bf16_bits(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// ---------------------------------------------------------------------------
// the row quantizer

constexpr int RQ_THREADS = 256;

// Eight values of a row from element `at` on; zeros behind n.
template <int SRC>
__device__ __forceinline__ void load8(const void* row, int at, int n, float (&v)[8]) {
  if (at + 8 <= n) {
    if (SRC == QR_BF16) {
      const u16x8_any h = *reinterpret_cast<const u16x8_any*>(reinterpret_cast<const uint16_t*>(row) + at);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = bf16_value(h[i]);
    } else {
      const f32x4_any* p = reinterpret_cast<const f32x4_any*>(reinterpret_cast<const float*>(row) + at);
      const f32x4_any a = p[0], b = p[1];
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
// Bound by one pass over memory: 8192 rows of 4096 bf16 values in 21 us, 4.8
// TB/s; a single row in 2.2 us, the time of its dependent loads.
template <int SRC, int KEEP>
__global__ __launch_bounds__(RQ_THREADS) void k_quantize_rows_i8(const void* __restrict__ x, int n, int64_t x_stride,
                                                                 int64_t row_bytes, int8_t* __restrict__ codes,
                                                                 float* __restrict__ scales) {
  __shared__ uint32_t wave_max[RQ_THREADS / WAVE];
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x;
  constexpr int ESIZE = SRC == QR_BF16 ? 2 : 4;
  const uint8_t* row = reinterpret_cast<const uint8_t*>(x) + r * x_stride * ESIZE;
  const int n_vec = (int)(row_bytes >> 3);
  float keep[KEEP][8];
  // magnitudes compare as integers, and a NaN or an infinity beats every
  // finite value there
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    load8<SRC>(row, (tid + k * RQ_THREADS) * 8, n, keep[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t m = __builtin_bit_cast(uint32_t, keep[k][i]) & 0x7fffffffu;
      top = m > top ? m : top;
    }
  }
  for (int g = tid + KEEP * RQ_THREADS; g < n_vec; g += RQ_THREADS) {
    float v[8];
    load8<SRC>(row, g * 8, n, v);
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
    load8<SRC>(row, g * 8, n, v);
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

// Which tile a workgroup takes. Workgroups are dealt to the 8 XCDs in turn;
// each XCD gets a run of neighbouring tiles, so that its L2 holds what they
// share, and walks it in bands of GROUP_T token tiles.
constexpr int XCDS = 8;
constexpr int GROUP_T = 4;

__device__ __forceinline__ void tile_of(uint32_t block, int out_tiles, int tok_tiles, int& bo, int& bt) {
  const int n = out_tiles * tok_tiles;
  const int xcd = (int)(block % XCDS), at = (int)(block / XCDS);
  const int each = n / XCDS, extra = n % XCDS;
  const int id = xcd * each + (xcd < extra ? xcd : extra) + at;
  const int band = id / (GROUP_T * out_tiles), in_band = id % (GROUP_T * out_tiles);
  const int width = tok_tiles - band * GROUP_T < GROUP_T ? tok_tiles - band * GROUP_T : GROUP_T;
  bt = band * GROUP_T + in_band % width;
  bo = in_band / width;
}

template <int DST>
__device__ __forceinline__ void store_one(void* y, int64_t at, float v) {
  if (DST == QR_BF16) reinterpret_cast<uint16_t*>(y)[at] = bf16_bits(v);
  else reinterpret_cast<float*>(y)[at] = v;
}

// A token's scale as xd * back: above 2^96 it is lowered by 2^32, so that a sum
// (up to 2^31) times it does not overflow before the channel's scale comes.
// Powers of two round nothing (8192 tokens, 11008 x 4096: 453 -> 459 us). At
// the other end a whole number times a scale loses no bits.
struct TokenScale {
  float d, back;
};

__device__ __forceinline__ TokenScale token_scale(float xd) {
  const bool high = __builtin_fabsf(xd) > 0x1p96f;
  return {high ? xd * 0x1p-32f : xd, high ? 0x1p32f : 1.0f};
}

__device__ __forceinline__ float scaled(int sum, const TokenScale& xd, float wd, float bias) {
  return (((float)sum * xd.d) * wd) * xd.back + bias;
}

// Stores four neighbouring channels of one token.
template <int DST>
__device__ __forceinline__ void store_four(const Product& p, int tok, int o, const i32x4& sum, const TokenScale& xd) {
  const int64_t at = (int64_t)tok * p.y_stride + o;
  if (o + 4 <= p.n_out) {
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = scaled(sum[e], xd, p.wd[o + e], p.bias ? p.bias[o + e] : 0.0f);
    if (DST == QR_BF16)
      *reinterpret_cast<u16x4_any*>(reinterpret_cast<uint16_t*>(p.y) + at) =
          u16x4_any{bf16_bits(v[0]), bf16_bits(v[1]), bf16_bits(v[2]), bf16_bits(v[3])};
    else
      *reinterpret_cast<f32x4_any*>(reinterpret_cast<float*>(p.y) + at) = f32x4_any{v[0], v[1], v[2], v[3]};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (o + e < p.n_out) store_one<DST>(p.y, at + e, scaled(sum[e], xd, p.wd[o + e], p.bias ? p.bias[o + e] : 0.0f));
  }
}

// Few tokens: 16 channels x 16 * TT tokens per workgroup, the sum split over
// its waves in chunks of 128 values, every operand loaded straight into the
// registers that the matrix instruction reads (row li, 16 bytes at 16 lk). The
// weights pass the chip once: bound by their bytes (16 tokens, 11008 x 4096:
// 14 us, 3.3 TB/s; one token, 4096 x 4096: 5.4 us). From some 24 tokens on
// every workgroup's reading of the tokens costs more, and tiles in LDS win.
constexpr int F_WAVES = 8;
constexpr int F_BATCH = 4;   // chunks of a wave whose loads are in flight together

template <int DST, int TT>
__global__ __launch_bounds__(F_WAVES* WAVE) void k_matmul_i8_few(Product p) {
  __shared__ i32x4 part[F_WAVES][TT][WAVE];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int li = lane & 15, lk = lane >> 4;
  const int out_tiles = (p.n_out + 15) / 16;
  const int o0 = (int)(blockIdx.x % out_tiles) * 16, t0 = (int)(blockIdx.x / out_tiles) * 16 * TT;
  // rows behind the last repeat it: their results are not stored
  const int wr = o0 + li < p.n_out ? o0 + li : p.n_out - 1;
  const int8_t* w = p.w + (int64_t)wr * p.row_bytes + 16 * lk;
  const int8_t* x[TT];
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int xr = t0 + 16 * j + li < p.n_tok ? t0 + 16 * j + li : p.n_tok - 1;
    x[j] = p.x + (int64_t)xr * p.row_bytes + 16 * lk;
  }
  const int chunks = p.row_bytes / 128;
  i32x4 acc[TT] = {};
  for (int c0 = wave; c0 < chunks; c0 += F_WAVES * F_BATCH) {
    i32x4 a[F_BATCH][2], b[F_BATCH][2][TT];
#pragma unroll
    for (int u = 0; u < F_BATCH; ++u) {
      const int c = c0 + u * F_WAVES < chunks ? c0 + u * F_WAVES : c0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        a[u][h] = *reinterpret_cast<const i32x4*>(w + c * 128 + 64 * h);
#pragma unroll
        for (int j = 0; j < TT; ++j) b[u][h][j] = *reinterpret_cast<const i32x4*>(x[j] + c * 128 + 64 * h);
      }
    }
#pragma unroll
    for (int u = 0; u < F_BATCH; ++u) {
      if (c0 + u * F_WAVES < chunks) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < TT; ++j)
            acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u][h], b[u][h][j], acc[j], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < TT; ++j) part[wave][j][lane] = acc[j];
  __syncthreads();
  if (wave < TT) {
    i32x4 sum = part[0][wave][lane];
#pragma unroll
    for (int v = 1; v < F_WAVES; ++v) sum += part[v][wave][lane];
    const int tok = t0 + 16 * wave + li;
    if (tok < p.n_tok) store_four<DST>(p, tok, o0 + 4 * lk, sum, token_scale(p.xd[tok]));
  }
}

// Many tokens: a tile of 64 NI channels x 64 NJ tokens per workgroup, a
// quarter of it per wave, 128 values of the sum per step through LDS. The
// weights are the matrix instruction's left operand: a lane then ends with
// runs of four neighbouring channels of one token.
//
// A step is four products of 32 values. While one is multiplied, the operands
// of the next come in from LDS; during the first three the next step's tile
// is written to the other LDS buffer and the one after that is asked for from
// memory. One barrier a step, before the fourth: it follows the last read of
// this tile and the writes of the next.
//
// In LDS the 16-byte piece c of row r lies at r * 128 + (c ^ (r / 2 % 8)) * 16:
// sixteen lanes that take one piece of neighbouring rows meet all banks.
//
// 32x32x32 products: with 16x16x64 ones the compiler moved 350 accumulators a
// step between registers. 8192^3: 1940 to 2130 TOP/s by card (a library product
// 2270 to 2510); 8192 x 11008 x 4096: 446 to 477 us. With the loads and stores
// not dealt between the products 8192^3 took 17% longer, with the loads right
// behind the stores 10%. The small tiles, several to a CU, keep loads early
// (11% slower otherwise).
//
// KS parts of a workgroup take every KS-th step, each with its own LDS, and
// add their sums up at the end: where there are few tiles a CU then has
// 8 or 16 waves at work on one.
template <int DST, int NI, int NJ, int KS>
__global__ __launch_bounds__(256 * KS) __attribute__((amdgpu_waves_per_eu(NI * NJ > 8 ? 1 : 2))) void k_matmul_i8_tile(
    Product p, int out_tiles, int tok_tiles) {
  constexpr int TO = 64 * NI, TT = 64 * NJ;
  constexpr bool LATE = NI * NJ > 8;   // ask for a tile late, between products that hide it
  __shared__ __attribute__((aligned(16))) int8_t all_lds[KS][2][(TO + TT) * 128];
  const int part = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  int8_t(*lds)[(TO + TT) * 128] = all_lds[part];
  const int tid = threadIdx.x & 255, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 31, lh = lane >> 5;
  int bo, bt;
  tile_of(blockIdx.x, out_tiles, tok_tiles, bo, bt);
  const int o0 = bo * TO, t0 = bt * TT;
  const int wo = (wave & 1) * (32 * NI), wt = (wave >> 1) * (32 * NJ);
  const int8_t* wbase = p.w + (int64_t)o0 * p.row_bytes;
  const int8_t* xbase = p.x + (int64_t)t0 * p.row_bytes;
  // rows behind the last repeat it: their results are not stored
  constexpr int NQ = 2 * NI + 2 * NJ;   // 32-row pieces of the tile: weights, then tokens
  const int lr = tid >> 3, lc = (tid & 7) * 16;
  uint32_t off[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int r = lr + 32 * (q < 2 * NI ? q : q - 2 * NI);
    const int last = q < 2 * NI ? p.n_out - 1 - o0 : p.n_tok - 1 - t0;
    off[q] = (uint32_t)(r < last ? r : last) * (uint32_t)p.row_bytes + lc;
  }
  const int put = lr * 128 + ((lc >> 4) ^ ((lr >> 1) & 7)) * 16;
  i32x4 raw[NQ];
  auto load = [&](int q, int64_t at) {
    raw[q] = *reinterpret_cast<const i32x4*>((q < 2 * NI ? wbase : xbase) + at + off[q]);
  };
  auto store = [&](int q, int8_t* buf) { *reinterpret_cast<i32x4*>(buf + put + q * 32 * 128) = raw[q]; };
  i32x4 a[2][NI], b[2][NJ];
  int get[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) get[k] = li * 128 + ((2 * k + lh) ^ ((li >> 1) & 7)) * 16;
  auto read = [&](const int8_t* buf, int k, i32x4(&ra)[NI], i32x4(&rb)[NJ]) {
#pragma unroll
    for (int i = 0; i < NI; ++i) ra[i] = *reinterpret_cast<const i32x4*>(buf + wo * 128 + get[k] + i * 32 * 128);
#pragma unroll
    for (int j = 0; j < NJ; ++j) rb[j] = *reinterpret_cast<const i32x4*>(buf + (TO + wt) * 128 + get[k] + j * 32 * 128);
  };
  i32x16 acc[NI][NJ] = {};
  // steps part, part + KS, ... are this part's; one behind the last is not used
  const int all = p.row_bytes / 128, steps = (all + KS - 1) / KS;
  auto at_step = [&](int s) { return (int64_t)(s * KS + part < all ? s * KS + part : all - 1) * 128; };
#pragma unroll
  for (int q = 0; q < NQ; ++q) load(q, at_step(0));
#pragma unroll
  for (int q = 0; q < NQ; ++q) store(q, lds[0]);
#pragma unroll
  for (int q = 0; q < NQ; ++q) load(q, at_step(1));
  __syncthreads();
  read(lds[0], 0, a[0], b[0]);
  for (int s = 0; s < steps; ++s) {
    const int8_t* cur = lds[s & 1];
    int8_t* nxt = lds[(s + 1) & 1];
    const int64_t ahead = at_step(s + 2);
    const bool mine = KS == 1 || s * KS + part < all;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k == 3) __syncthreads();
      read(k == 3 ? nxt : cur, (k + 1) & 3, a[(k + 1) & 1], b[(k + 1) & 1]);
      if (k < 3) {
#pragma unroll
        for (int q = k * NQ / 3; q < (k + 1) * NQ / 3; ++q) {
          store(q, nxt);
          if (!LATE) load(q, ahead);
        }
      }
      if (LATE && k > 0) {   // behind the stores of the same pieces
#pragma unroll
        for (int q = (k - 1) * NQ / 4; q < (k == 3 ? NQ : k * NQ / 4); ++q) load(q, ahead);
      }
      if (!mine) continue;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[k & 1][i], b[k & 1][j], acc[i][j], 0, 0, 0);
      // memory instructions between the products, so that the matrix core does
      // not wait for an issue slot
#pragma unroll
      for (int q = 0; LATE && q < NI * NJ; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                       // product
        if (q < NI + NJ) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);      // LDS read
        else if (k < 3) __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);       // LDS write
        if (q >= NI + NJ && k > 0 && (k == 3 || q % 2)) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);   // load
      }
    }
  }
  if constexpr (KS > 1) {
    // the parts' sums added up, one part after the other in the same LDS
    i32x16* sums = reinterpret_cast<i32x16*>(all_lds);   // [wave][tile][lane]
    static_assert(4 * NI * NJ * 64 * 64 <= (int)sizeof(all_lds), "the sums fit");
    for (int from = 1; from < KS; ++from) {
      __syncthreads();
      if (part == from) {
#pragma unroll
        for (int n = 0; n < NI * NJ; ++n) sums[(wave * NI * NJ + n) * 64 + lane] = acc[n / NJ][n % NJ];
      }
      __syncthreads();
      if (part == 0) {
#pragma unroll
        for (int n = 0; n < NI * NJ; ++n) acc[n / NJ][n % NJ] += sums[(wave * NI * NJ + n) * 64 + lane];
      }
    }
    if (part != 0) return;
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int tok = t0 + wt + 32 * j + li;
    if (tok >= p.n_tok) continue;
    const TokenScale xd = token_scale(p.xd[tok]);
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        store_four<DST>(p, tok, o0 + wo + 32 * i + 2 * e + 4 * lh,
                        i32x4{acc[i][j][e], acc[i][j][e + 1], acc[i][j][e + 2], acc[i][j][e + 3]}, xd);
  }
}

template <int DST, int TT>
int launch_few(const Product& p, hipStream_t s) {
  const int64_t tiles = (int64_t)((p.n_out + 15) / 16) * ((p.n_tok + 16 * TT - 1) / (16 * TT));
  if (tiles > UINT32_MAX / (F_WAVES * WAVE)) return qr_fail(QR_EOVERFLOW, "n_out and n_tok need too many tiles for one launch");
  hipLaunchKernelGGL((k_matmul_i8_few<DST, TT>), dim3((uint32_t)tiles), dim3(F_WAVES * WAVE), 0, s, p);
  return qr_check_launch("k_matmul_i8_few");
}

template <int DST, int NI, int NJ, int KS>
int launch_tile(const Product& p, hipStream_t s) {
  const int out_tiles = (p.n_out + 64 * NI - 1) / (64 * NI), tok_tiles = (p.n_tok + 64 * NJ - 1) / (64 * NJ);
  const int64_t tiles = (int64_t)out_tiles * tok_tiles;
  if (tiles > UINT32_MAX / (256 * KS)) return qr_fail(QR_EOVERFLOW, "n_out and n_tok need too many tiles for one launch");
  hipLaunchKernelGGL((k_matmul_i8_tile<DST, NI, NJ, KS>), dim3((uint32_t)tiles), dim3(256 * KS), 0, s, p, out_tiles, tok_tiles);
  return qr_check_launch("k_matmul_i8_tile");
}

int64_t tiles_of(const Product& p, int out, int tok) {
  return (int64_t)((p.n_out + out - 1) / out) * ((p.n_tok + tok - 1) / tok);
}

// The tile: as large as leaves the chip's 256 CUs a workgroup each (an LDS
// byte then serves more products), and below that the sum split inside a
// workgroup, so that a CU has 8 or 16 waves at work. Measured, us (channels x
// values 4096 x 4096 unless said), the choice first:
//   16 tokens            k_few 1: 11      64x64 in four parts: 14
//   24 x 11008 channels  64x64 in four: 15     k_few 2: 23
//   48 tokens            k_few 4: 12           64x64 in four: 14
//   64 x 11008           64x64 in four: 17     k_few 4: 34
//   128 x 11008          64x128 in two: 21     64x64 in four: 29
//   512                  64x128 in two: 20     64x64 in four: 27
//   1024                 128x128 in two: 29    64x128 in two: 37
//   1500                 128x128: 44           128x128 in two: 53
//   4096                 256x256: 82           128x128: 96
//   700 x 11008 (129 tiles of 256x256)         128x128: 70    256x256: 74
template <int DST>
int launch_product(const Product& p, hipStream_t s) {
  constexpr int64_t CUS = 256;
  if (p.n_tok <= 16) return launch_few<DST, 1>(p, s);
  const int64_t t64 = tiles_of(p, 64, 64);
  if (p.n_tok <= 64 && t64 < 96) {   // few channels too
    if (p.n_tok > 32 && tiles_of(p, 16, 64) >= CUS) return launch_few<DST, 4>(p, s);
    return launch_few<DST, 2>(p, s);
  }
  if (t64 <= CUS) return launch_tile<DST, 1, 1, 4>(p, s);
  if (tiles_of(p, 64, 128) <= CUS) return launch_tile<DST, 1, 2, 2>(p, s);
  if (tiles_of(p, 128, 128) <= CUS) return launch_tile<DST, 2, 2, 2>(p, s);
  // 256x256 where the last round of workgroups does not leave too many idle
  const int64_t t256 = tiles_of(p, 256, 256), rounds = (t256 + CUS - 1) / CUS;
  if (t256 * 100 >= rounds * CUS * 65) return launch_tile<DST, 4, 4, 1>(p, s);
  return launch_tile<DST, 2, 2, 1>(p, s);
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
