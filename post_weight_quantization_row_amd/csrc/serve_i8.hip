// serve_i8.hip -- gfx950 kernels and C-ABI of 8-bit rows with one scale each
// and of their product (declared in serve/qrow_i8.h).

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "qr_internal.h"
#include "qrow.h"
#include "serve/qrow_i8.h"
#include "serve_internal.h"

namespace {

using namespace serve;

typedef int i32x16 __attribute__((ext_vector_type(16)));
constexpr int ROW_ALIGN = 128;   // bytes: qr_i8_row_bytes

// ---------------------------------------------------------------------------
// the row quantizer

constexpr int RQ_THREADS = 256;

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
  const CodeScale c = code_scale(top);
  int8_t* out = codes + r * row_bytes;
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    const int g = tid + k * RQ_THREADS;
    if (g < n_vec) *reinterpret_cast<u32x2*>(out + (int64_t)g * 8) = c.finite ? pack_codes(keep[k], c.inv) : u32x2{0, 0};
  }
  for (int g = tid + KEEP * RQ_THREADS; g < n_vec; g += RQ_THREADS) {
    float v[8];
    load8<SRC>(row, g * 8, n, v);
    *reinterpret_cast<u32x2*>(out + (int64_t)g * 8) = c.finite ? pack_codes(v, c.inv) : u32x2{0, 0};
  }
  if (tid == 0) scales[r] = c.d;
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

// What comes behind the sums (EPI): nothing but scales and bias, an activation
// and a residual, or those and the gate's second product.
enum { PLAIN, ACT, GATED };

struct Epilogue {
  const int8_t* up;
  const float* upd;
  const float* up_bias;
  const void* residual;
  int64_t residual_stride;
  int act;
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

template <int SRC>
__device__ __forceinline__ float load_one(const void* x, int64_t at) {
  return SRC == QR_BF16 ? bf16_value(reinterpret_cast<const uint16_t*>(x)[at]) : reinterpret_cast<const float*>(x)[at];
}

// Scales and biases of four neighbouring channels; the last one's behind it.
template <int EPI>
struct Channels {
  float wd[4], bias[4], upd[4], up_bias[4];

  __device__ __forceinline__ Channels(const Product& p, const Epilogue& ep, int o) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = o + e < p.n_out ? o + e : p.n_out - 1;
      wd[e] = p.wd[c];
      bias[e] = p.bias ? p.bias[c] : 0.0f;
      upd[e] = EPI == GATED ? ep.upd[c] : 0.0f;
      up_bias[e] = EPI == GATED && ep.up_bias ? ep.up_bias[c] : 0.0f;
    }
  }
};

// Four neighbouring channels of some tokens: sums (up: the gate's second ones),
// token and its scale. A token of -1 is none.
struct Four {
  i32x4 sum, up;
  TokenScale d;
  int tok;
};

template <int DST, int EPI, int N>
__device__ __forceinline__ void store_fours(const Product& p, const Epilogue& ep, const Channels<EPI>& c, int o, const Four (&f)[N]) {
  const bool whole = o + 4 <= p.n_out;
  float v[4 * N];
#pragma unroll
  for (int t = 0; t < N; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * t + e] = scaled(f[t].sum[e], f[t].d, c.wd[e], c.bias[e]);
  if (EPI != PLAIN) activate(ep.act, v);
#pragma unroll
  for (int t = 0; t < N; ++t) {
    if (f[t].tok < 0) continue;
    const int64_t at = (int64_t)f[t].tok * p.y_stride + o, from = (int64_t)f[t].tok * ep.residual_stride + o;
    float u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      u[e] = v[4 * t + e];
      if (EPI == GATED) u[e] *= scaled(f[t].up[e], f[t].d, c.upd[e], c.up_bias[e]);
    }
    if (EPI != PLAIN && ep.residual) {
      if (whole && DST == QR_BF16) {
        const u16x4_any r = *reinterpret_cast<const u16x4_any*>(reinterpret_cast<const uint16_t*>(ep.residual) + from);
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] += bf16_value(r[e]);
      } else if (whole) {
        const f32x4_any r = *reinterpret_cast<const f32x4_any*>(reinterpret_cast<const float*>(ep.residual) + from);
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] += r[e];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (o + e < p.n_out) u[e] += load_one<DST>(ep.residual, from + e);
      }
    }
    if (whole && DST == QR_BF16) {
      *reinterpret_cast<u16x4_any*>(reinterpret_cast<uint16_t*>(p.y) + at) =
          u16x4_any{bf16_bits(u[0]), bf16_bits(u[1]), bf16_bits(u[2]), bf16_bits(u[3])};
    } else if (whole) {
      *reinterpret_cast<f32x4_any*>(reinterpret_cast<float*>(p.y) + at) = f32x4_any{u[0], u[1], u[2], u[3]};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (o + e < p.n_out) store_one<DST>(p.y, at + e, u[e]);
    }
  }
}

// The same without an epilogue, where the scales are loaded as they are needed.
template <int DST>
__device__ __forceinline__ void store_plain(const Product& p, int tok, int o, const i32x4& sum, const TokenScale& xd) {
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
// registers that the matrix instruction reads (row li, 16 bytes at 16 lk; whole
// lines of the weights, turned in registers). The weights pass the chip once:
// bound by their bytes (16 tokens, 11008 x 4096: 14.2 to 15.0 us by card, 3.0 to 3.2
// TB/s; one token, 4096 x 4096: 5.4 us). From some 24 tokens on
// every workgroup's reading of the tokens costs more, and tiles in LDS win.
constexpr int F_WAVES = 8;
// Chunks of a wave whose loads are in flight together: with a gate, which has
// twice the rows, two of them in 64 registers leave room for four workgroups on
// a CU (one token, 11008 x 4096 gated: 19.1 us, four 21.9; without a gate, 4096
// x 4096: two 6.3 us, four 5.5).
template <int EPI>
constexpr int few_batch() { return EPI == GATED ? 2 : 4; }

template <int DST, int TT, int EPI>
__global__ __launch_bounds__(F_WAVES* WAVE) void k_matmul_i8_few(Product p, Epilogue ep) {
  constexpr int G = EPI == GATED ? 2 : 1;   // weight rows per channel: gate and up
  constexpr int F_BATCH = few_batch<EPI>();
  __shared__ i32x4 part[F_WAVES][G][TT][WAVE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lk = lane >> 4;
  const int out_tiles = (p.n_out + 15) / 16;
  const int o0 = (int)(blockIdx.x % out_tiles) * 16, t0 = (int)(blockIdx.x / out_tiles) * 16 * TT;
  // rows behind the last repeat it: their results are not stored
  const int w_last = p.n_out - o0 < 16 ? p.n_out - 1 - o0 : 15, x_last = p.n_tok - t0 < 16 * TT ? p.n_tok - 1 - t0 : 16 * TT - 1;
  const uint32_t rb = (uint32_t)p.row_bytes;
  Buffer w[G];
#pragma unroll
  for (int g = 0; g < G; ++g) w[g] = buffer_of((g ? ep.up : p.w) + (int64_t)o0 * p.row_bytes, (uint32_t)(w_last + 1) * rb);
  const Buffer xs = buffer_of(p.x + (int64_t)t0 * p.row_bytes, (uint32_t)(x_last + 1) * rb);
  uint32_t at[2], x[TT];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = 8 * h + (li & 7);
    at[h] = (uint32_t)(r < w_last ? r : w_last) * rb + 64 * (li >> 3) + 16 * lk;
  }
#pragma unroll
  for (int j = 0; j < TT; ++j) x[j] = 16 * j + li <= x_last ? (uint32_t)(16 * j + li) * rb + 16 * lk : NOWHERE;
  const int chunks = p.row_bytes / 128;
  i32x4 acc[G][TT] = {};
  for (int c0 = wave; c0 < chunks; c0 += F_WAVES * F_BATCH) {
    i32x4 a[F_BATCH][G][2], b[F_BATCH][2][TT];
#pragma unroll
    for (int u = 0; u < F_BATCH; ++u) {
      const int c = (c0 + u * F_WAVES < chunks ? c0 + u * F_WAVES : c0) * 128;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // (two workgroups of 32 tokens may read the same weights)
#pragma unroll
        for (int g = 0; g < G; ++g) a[u][g][h] = TT == 2 ? load16(w[g], at[h], c) : load16_once(w[g], at[h], c);
#pragma unroll
        for (int j = 0; j < TT; ++j) b[u][h][j] = load16(xs, x[j], c + 64 * h);
      }
    }
#pragma unroll
    for (int u = 0; u < F_BATCH; ++u) {
      if (c0 + u * F_WAVES < chunks) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          turn(a[u][g][0], a[u][g][1]);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < TT; ++j)
              acc[g][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u][g][h], b[u][h][j], acc[g][j], 0, 0, 0);
        }
      }
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int j = 0; j < TT; ++j) part[wave][g][j][lane] = acc[g][j];
  __syncthreads();
  if (wave < TT) {
    i32x4 sum[2];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      sum[g] = part[0][g][wave][lane];
#pragma unroll
      for (int v = 1; v < F_WAVES; ++v) sum[g] += part[v][g][wave][lane];
    }
    const int tok = t0 + 16 * wave + li;
    if (tok >= p.n_tok) return;
    if constexpr (EPI == PLAIN) store_plain<DST>(p, tok, o0 + 4 * lk, sum[0], token_scale(p.xd[tok]));
    else store_fours<DST, EPI, 1>(p, ep, Channels<EPI>(p, ep, o0 + 4 * lk), o0 + 4 * lk, {{sum[0], sum[G - 1], token_scale(p.xd[tok]), tok}});
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
// step between registers. 8192^3: 2020 to 2200 TOP/s by card and codes (a library
// product on the same card 2000 to 2310); 8192 x 11008 x 4096: 380 to 410 us; with
// a gate 750 to 820, in which the matrix cores are busy for 48% of the clocks (they
// alone, fed from registers, reach 3050 to 3300 TOP/s). The loop itself passes at
// 2700 (sums of 512 and of 4096 values compared); 30% of the gate's time is the
// epilogue, during which its CU multiplies nothing. Workgroups that go on to a next
// tile, its first steps asked for before the epilogue: no faster. With the loads and
// stores not dealt between the products 8192^3 took 17% longer, with the loads
// right behind the stores 10%. The small tiles, several to a CU, keep loads early
// (11% slower otherwise).
//
// KS parts of a workgroup take every KS-th step, each with its own LDS, and
// add their sums up at the end: where there are few tiles a CU then has
// 8 or 16 waves at work on one.
//
// With a gate a piece of 32 weight rows is 16 of gate and the same 16 channels'
// of up: a lane's accumulators e and e + 8 are then the two sums of a channel,
// and a tile has half as many channels.
template <int DST, int NI, int NJ, int KS, int EPI>
__global__ __launch_bounds__(256 * KS) __attribute__((amdgpu_waves_per_eu(NI * NJ > 8 ? 1 : 2))) void k_matmul_i8_tile(
    Product p, Epilogue ep, int out_tiles, int tok_tiles) {
  constexpr int TO = 64 * NI, TT = 64 * NJ;
  constexpr bool LATE = NI * NJ > 8;   // ask for a tile late, between products that hide it
  __shared__ __attribute__((aligned(16))) int8_t all_lds[KS][2][(TO + TT) * 128];
  const int part = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  int8_t(*lds)[(TO + TT) * 128] = all_lds[part];
  const int tid = threadIdx.x & 255, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 31, lh = lane >> 5;
  int bo, bt;
  tile_of(blockIdx.x, out_tiles, tok_tiles, bo, bt);
  constexpr int PIECE = EPI == GATED ? 16 : 32;   // channels of 32 weight rows
  const int o0 = bo * (2 * NI * PIECE), t0 = bt * TT;
  const int wo = (wave & 1) * (32 * NI), wt = (wave >> 1) * (32 * NJ);
  // (the lanes of a wave stage eight rows: gate's or up's)
  const int8_t* wbase = (EPI == GATED && wave >= 2 ? ep.up : p.w) + (int64_t)o0 * p.row_bytes;
  const int8_t* xbase = p.x + (int64_t)t0 * p.row_bytes;
  // rows behind the last repeat it: their results are not stored
  constexpr int NQ = 2 * NI + 2 * NJ;   // 32-row pieces of the tile: weights, then tokens
  const int lr = tid >> 3, lc = (tid & 7) * 16;
  uint32_t off[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int r = q < 2 * NI ? lr % PIECE + PIECE * q : lr + 32 * (q - 2 * NI);
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
  {
    i32x4 first[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      load(q, at_step(0));
      first[q] = raw[q];
    }
#pragma unroll
    for (int q = 0; q < NQ; ++q) load(q, at_step(1));
#pragma unroll
    for (int q = 0; q < NQ; ++q) *reinterpret_cast<i32x4*>(lds[0] + put + q * 32 * 128) = first[q];
  }
  float xd[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int tok = t0 + wt + 32 * j + li;
    xd[j] = p.xd[tok < p.n_tok ? tok : p.n_tok - 1];
  }
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
    __syncthreads();   // the sums have been read
    if (part != 0) return;
  } else {
    __syncthreads();   // the last tile has been read
  }
  // 32 tokens at a time through the wave's own part of LDS: the epilogue is then
  // one short loop (unrolled over the accumulators it was too long for the
  // compiler to keep them in registers), a lane keeps its four channels, and a
  // token's are stored side by side. Behind a token's sums lies its scale.
  constexpr int W = 32 * NI, PITCH = W + 4, FOURS = W / (EPI == GATED ? 8 : 4), TOKENS = 64 / FOURS, AT_ONCE = 2;
  static_assert(4 * 32 * PITCH * 4 <= (int)sizeof(all_lds), "the waves' sums fit");
  int* sums = reinterpret_cast<int*>(all_lds) + wave * (32 * PITCH);
  const int four = lane % FOURS, piece = four * 4 / PIECE, o = o0 + (wo / 32 + piece) * PIECE + four * 4 % PIECE;
  const Channels<EPI> channels(p, ep, o < p.n_out ? o : p.n_out - 1);
  const int* from = sums + (lane / FOURS) * PITCH + 32 * piece + four * 4 % PIECE;
  const int* scales = sums + (lane / FOURS) * PITCH + W;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int first = t0 + wt + 32 * j;
    if (first >= p.n_tok) break;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *reinterpret_cast<i32x4*>(sums + li * PITCH + 32 * i + 2 * e + 4 * lh) =
            i32x4{acc[i][j][e], acc[i][j][e + 1], acc[i][j][e + 2], acc[i][j][e + 3]};
    if (lh == 0) *reinterpret_cast<TokenScale*>(sums + li * PITCH + W) = token_scale(xd[j]);
    wave_sync();
#pragma unroll 1
    for (int t = 0; t < 32; t += AT_ONCE * TOKENS) {
      Four f[AT_ONCE];
#pragma unroll
      for (int u = 0; u < AT_ONCE; ++u) {
        const int r = t + u * TOKENS, tok = first + r + lane / FOURS;
        f[u] = {*reinterpret_cast<const i32x4*>(from + r * PITCH), *reinterpret_cast<const i32x4*>(from + r * PITCH + (EPI == GATED ? 16 : 0)),
                *reinterpret_cast<const TokenScale*>(scales + r * PITCH), tok < p.n_tok && o < p.n_out ? tok : -1};
      }
      store_fours<DST, EPI, AT_ONCE>(p, ep, channels, o, f);
    }
    wave_sync();
  }
}

template <int DST, int TT, int EPI>
int launch_few(const Product& p, const Epilogue& ep, hipStream_t s) {
  const int64_t tiles = (int64_t)((p.n_out + 15) / 16) * ((p.n_tok + 16 * TT - 1) / (16 * TT));
  if (tiles > UINT32_MAX / (F_WAVES * WAVE)) return qr_fail(QR_EOVERFLOW, "n_out and n_tok need too many tiles for one launch");
  hipLaunchKernelGGL((k_matmul_i8_few<DST, TT, EPI>), dim3((uint32_t)tiles), dim3(F_WAVES * WAVE), 0, s, p, ep);
  return qr_check_launch("k_matmul_i8_few");
}

template <int DST, int NI, int NJ, int KS, int EPI>
int launch_tile(const Product& p, const Epilogue& ep, hipStream_t s) {
  constexpr int TO = EPI == GATED ? 32 * NI : 64 * NI;   // channels of a tile
  const int out_tiles = (p.n_out + TO - 1) / TO, tok_tiles = (p.n_tok + 64 * NJ - 1) / (64 * NJ);
  const int64_t tiles = (int64_t)out_tiles * tok_tiles;
  if (tiles > UINT32_MAX / (256 * KS)) return qr_fail(QR_EOVERFLOW, "n_out and n_tok need too many tiles for one launch");
  hipLaunchKernelGGL((k_matmul_i8_tile<DST, NI, NJ, KS, EPI>), dim3((uint32_t)tiles), dim3(256 * KS), 0, s, p, ep,
                     out_tiles, tok_tiles);
  return qr_check_launch("k_matmul_i8_tile");
}

// Tiles of `out` weight rows x `tok` tokens; a gate has two rows per channel.
template <int EPI>
int64_t tiles_of(const Product& p, int out, int tok) {
  const int64_t rows = EPI == GATED ? 2 * (int64_t)p.n_out : p.n_out;
  return ((rows + out - 1) / out) * ((p.n_tok + tok - 1) / tok);
}

// The tile: as large as leaves the chip's 256 CUs a workgroup each (an LDS
// byte then serves more products), and below that the sum split inside a
// workgroup, so that a CU has 8 or 16 waves at work. Measured, us (channels x
// values 4096 x 4096 unless said), the choice first:
//   16 tokens            k_few 1: 6.5     64x64 in four parts: 11
//   24 x 11008 channels  64x64 in four: 13     k_few 2: 18
//   48 tokens            k_few 4: 11           64x64 in four: 11
//   64 x 11008           64x64 in four: 13     k_few 4: 31
//   128 x 11008          64x128 in two: 17     64x64 in four: 23
//   512                  64x128 in two: 18     64x64 in four: 24
//   1024                 128x128 in two: 28    64x128 in two: 34
//   1500                 128x128: 43           128x128 in two: 48
//   2000 (128 tiles of 256x256)                128x128: 50    256x256: 57
//   700 x 11008 (129)    256x256: 53           128x128: 62
//   4096 (256)           256x256: 76           128x128: 93
//   4800 (304)           128x128: 106          256x256: 119
//   5800 (368)           256x256: 122          128x128: 129
template <int DST, int EPI>
int launch_product(const Product& p, const Epilogue& ep, hipStream_t s) {
  constexpr int64_t CUS = 256;
  if (p.n_tok <= 16) return launch_few<DST, 1, EPI>(p, ep, s);
  const int64_t t64 = tiles_of<EPI>(p, 64, 64);
  if (p.n_tok <= 64 && t64 < 96) {   // few channels too
    if (p.n_tok > 32 && tiles_of<EPI>(p, 16, 64) >= CUS) return launch_few<DST, 4, EPI>(p, ep, s);
    return launch_few<DST, 2, EPI>(p, ep, s);
  }
  if (t64 <= CUS) return launch_tile<DST, 1, 1, 4, EPI>(p, ep, s);
  if (tiles_of<EPI>(p, 64, 128) <= CUS) return launch_tile<DST, 1, 2, 2, EPI>(p, ep, s);
  if (tiles_of<EPI>(p, 128, 128) <= CUS) return launch_tile<DST, 2, 2, 2, EPI>(p, ep, s);
  // 256x256 where the last round of workgroups does not leave too many idle: a
  // single round may be half empty, since 128x128 needs a second one there
  const int64_t t256 = tiles_of<EPI>(p, 256, 256), rounds = (t256 + CUS - 1) / CUS;
  if (t256 * 100 > rounds * CUS * (rounds == 1 ? 50 : 65)) return launch_tile<DST, 4, 4, 1, EPI>(p, ep, s);
  return launch_tile<DST, 2, 2, 1, EPI>(p, ep, s);
}

template <int EPI>
int launch_to(int dst, const Product& p, const Epilogue& ep, hipStream_t s) {
  return dst == QR_BF16 ? launch_product<QR_BF16, EPI>(p, ep, s) : launch_product<QR_F32, EPI>(p, ep, s);
}

// The checks that both products share; QR_OK with *none set: nothing to do.
int check_product(const int8_t* w, const float* wd, const int8_t* x, const float* xd, const float* bias, int64_t n_out,
                  int64_t n_tok, int64_t n_in, int dst, const void* y, int64_t y_stride, bool* none) {
  *none = false;
  if (dst != QR_F32 && dst != QR_BF16) return qr_fail(QR_EINVAL_TYPE, "output type %d is not QR_F32 or QR_BF16", dst);
  if (qr_i8_row_bytes(n_in) == 0) return qr_fail(QR_EINVAL_SHAPE, "n_in=%lld must be in 1..%d", (long long)n_in, QR_I8_MAX_IN);
  if (n_out < 0 || n_tok < 0 || y_stride < n_out)
    return qr_fail(QR_EINVAL_SHAPE, "negative n_out or n_tok, or y_stride below n_out");
  *none = n_out == 0 || n_tok == 0;
  if (*none) return QR_OK;
  if (n_out > INT32_MAX - 256 || n_tok > INT32_MAX - 256 || y_stride > INT64_MAX / 4 / n_tok)
    return qr_fail(QR_EOVERFLOW, "n_out or n_tok too large");
  if (!w || !wd || !x || !xd || !y) return qr_fail(QR_EINVAL_PTR, "w, wd, x, xd and y must be non-NULL");
  if (!qr_aligned(w, 16) || !qr_aligned(x, 16) || !qr_aligned(wd, 4) || !qr_aligned(xd, 4) || !qr_aligned(bias, 4) ||
      !qr_aligned(y, dst == QR_BF16 ? 2 : 4))
    return qr_fail(QR_EINVAL_PTR, "codes must be 16-byte aligned, wd, xd, bias and y to their elements");
  return QR_OK;
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
  return qr_matmul_i8_ex(w, wd, x, xd, bias, nullptr, n_out, n_tok, n_in, dst, y, y_stride, stream);
}

int qr_matmul_i8_ex(const int8_t* w, const float* wd, const int8_t* x, const float* xd, const float* bias,
                    const qr_i8_epilogue* e, int64_t n_out, int64_t n_tok, int64_t n_in, int dst, void* y,
                    int64_t y_stride, void* stream) {
  qr_clear_error();
  bool none;
  const int rc = check_product(w, wd, x, xd, bias, n_out, n_tok, n_in, dst, y, y_stride, &none);
  if (rc != QR_OK) return rc;
  if (e && (e->act < QR_ACT_NONE || e->act > QR_ACT_GELU_TANH))
    return qr_fail(QR_EINVAL_TYPE, "activation %lld is not one of QR_ACT_*", (long long)e->act);
  if (e && e->residual && e->residual_stride < n_out) return qr_fail(QR_EINVAL_SHAPE, "residual_stride is below n_out");
  if (none) return QR_OK;
  const Product p = {w, x, wd, xd, bias, y, y_stride, (int)n_out, (int)n_tok, (int)qr_i8_row_bytes(n_in)};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (!e || (e->act == QR_ACT_NONE && !e->up && !e->residual)) return launch_to<PLAIN>(dst, p, Epilogue{}, s);
  if (e->up) {
    if (n_out > (INT32_MAX - 256) / 2) return qr_fail(QR_EOVERFLOW, "n_out or n_tok too large");
    if (!e->upd) return qr_fail(QR_EINVAL_PTR, "up needs upd");
    if (!qr_aligned(e->up, 16) || !qr_aligned(e->upd, 4) || !qr_aligned(e->up_bias, 4))
      return qr_fail(QR_EINVAL_PTR, "up must be 16-byte aligned, upd and up_bias to their elements");
  }
  if (e->residual) {
    const int64_t esize = dst == QR_BF16 ? 2 : 4;
    if (e->residual_stride > INT64_MAX / 4 / n_tok) return qr_fail(QR_EOVERFLOW, "residual_stride is too large");
    if (!qr_aligned(e->residual, (uintptr_t)esize)) return qr_fail(QR_EINVAL_PTR, "residual must be aligned to its elements");
    const bool in_place = e->residual == y && (n_tok == 1 || e->residual_stride == y_stride);
    if (!in_place && rows_meet(y, y_stride * esize, e->residual, e->residual_stride * esize, n_out * esize, n_tok))
      return qr_fail(QR_EINVAL_PTR, "y and residual must be the same rows or not overlap");
  }
  const Epilogue ep = {e->up, e->upd, e->up_bias, e->residual, e->residual_stride, (int)e->act};
  return e->up ? launch_to<GATED>(dst, p, ep, s) : launch_to<ACT>(dst, p, ep, s);
}

}  // extern "C"
