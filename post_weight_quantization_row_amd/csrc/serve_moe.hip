// serve_moe.hip -- gfx950 kernels and C-ABI of a mixture of experts in 8 bits:
// the router and the experts of a few tokens (declared in serve/qrow_moe.h).

#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "qr_internal.h"
#include "qrow.h"
#include "serve/qrow_moe.h"
#include "serve_internal.h"

namespace {

using namespace serve;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// the router

struct Route {
  const void* x;
  const void* w;
  const float* bias;
  double* logits;        // [splits][n_tok][n_experts]
  float* squares;        // of rough logits, sums over the rows: [splits][n_tok] of x, [splits][n_experts] of w
  int32_t* ids;
  float* weights;
  int64_t x_stride;
  int n_experts, n_tok, n_in, top_k, splits, score, renorm;
  float factor;
};

constexpr int R_CHUNK = 32;      // values of the sum that a wave takes at a time
constexpr int R_WAVES = 8;
constexpr int R_SPLITS = 8;      // at most

// Eight neighbouring values as they lie in memory.
template <int SRC>
struct Eight {
  u16x8_any v;
  __device__ __forceinline__ double get(int i) const { return (double)bf16_value(v[i]); }
};
template <>
struct Eight<QR_F32> {
  f32x4_any v[2];
  __device__ __forceinline__ double get(int i) const { return (double)v[i >> 2][i & 3]; }
};

template <int SRC>
__device__ __forceinline__ Eight<SRC> eight_at(const uint8_t* row, int at) {
  return *reinterpret_cast<const Eight<SRC>*>(row + (int64_t)at * (SRC == QR_BF16 ? 2 : 4));
}

// Logits: 16 TE experts x 16 TT tokens per workgroup, the sum split over its
// waves (and, with few tiles, over workgroups) in chunks of 32 values. Products
// of fp32 values are exact in 64 bits, and so are the 64-bit matrix
// instructions' operands: row li, element lk of each four. A lane loads eight
// neighbouring values and feeds them to eight instructions, both sides alike.
//
// With many tokens bound by the 64-bit matrix instructions: 2048 tokens, 256
// experts, 7168 values 127 us, 59 TFLOP/s (a large 64-bit library product: 71).
// Few tokens are the time of two dependent trips to memory (one token: 5.9 us).
template <int SRC, int WSRC, int TE, int TT>
__global__ __launch_bounds__(R_WAVES* WAVE) void k_route_logits(Route p, int expert_tiles, int token_tiles) {
  __shared__ f64x4 part[R_WAVES][TE][TT][WAVE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lk = lane >> 4;
  int block = (int)blockIdx.x;
  const int be = block % expert_tiles;
  block /= expert_tiles;
  const int bt = block % token_tiles, split = block / token_tiles;
  const uint8_t *xr[TT], *wr[TE];
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int t = (bt * TT + j) * 16 + li;
    xr[j] = reinterpret_cast<const uint8_t*>(p.x) + (int64_t)(t < p.n_tok ? t : p.n_tok - 1) * p.x_stride * (SRC == QR_BF16 ? 2 : 4);
  }
#pragma unroll
  for (int i = 0; i < TE; ++i) {
    const int e = (be * TE + i) * 16 + li;
    wr[i] = reinterpret_cast<const uint8_t*>(p.w) + (int64_t)(e < p.n_experts ? e : p.n_experts - 1) * p.n_in * (WSRC == QR_BF16 ? 2 : 4);
  }
  f64x4 acc[TE][TT] = {};
  struct Stage {
    Eight<WSRC> a[TE];
    Eight<SRC> b[TT];
  };
  // whole chunks first, then what is left of the row, for the wave whose turn it is
  const int chunks = p.n_in / R_CHUNK, step = R_WAVES * p.splits, from = split * R_WAVES + wave;
  pipeline<TE * TT == 1 ? 4 : 2, Stage>(from, chunks, step,
      [&](Stage& s, int k) {
#pragma unroll
        for (int i = 0; i < TE; ++i) s.a[i] = eight_at<WSRC>(wr[i], k * R_CHUNK + 8 * lk);
#pragma unroll
        for (int j = 0; j < TT; ++j) s.b[j] = eight_at<SRC>(xr[j], k * R_CHUNK + 8 * lk);
      },
      [&](Stage& s, int) {
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
          for (int i = 0; i < TE; ++i)
#pragma unroll
            for (int j = 0; j < TT; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f64_16x16x4f64(s.a[i].get(u), s.b[j].get(u), acc[i][j], 0, 0, 0);
      });
  if (p.n_in % R_CHUNK != 0 && chunks % step == from) {
    float a[TE][8], b[TT][8];
#pragma unroll
    for (int i = 0; i < TE; ++i) load8<WSRC>(wr[i], chunks * R_CHUNK + 8 * lk, p.n_in, a[i]);
#pragma unroll
    for (int j = 0; j < TT; ++j) load8<SRC>(xr[j], chunks * R_CHUNK + 8 * lk, p.n_in, b[j]);
#pragma unroll
    for (int u = 0; u < 8; ++u)
#pragma unroll
      for (int i = 0; i < TE; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f64_16x16x4f64((double)a[i][u], (double)b[j][u], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < TE; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) part[wave][i][j][lane] = acc[i][j];
  __syncthreads();
  for (int n = wave; n < TE * TT; n += R_WAVES) {
    const int i = n / TT, j = n % TT;
    f64x4 sum = part[0][i][j][lane];
#pragma unroll
    for (int v = 1; v < R_WAVES; ++v) sum += part[v][i][j][lane];
    const int t = (bt * TT + j) * 16 + li;
    if (t >= p.n_tok) continue;
    double* out = p.logits + ((int64_t)split * p.n_tok + t) * p.n_experts;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int e = (be * TE + i) * 16 + 4 * v + lk;
      if (e < p.n_experts) out[e] = sum[v];
    }
  }
}

// 64-bit values in the order of their keys: a NaN above everything, nothing
// (key 0) below.
__device__ __forceinline__ uint64_t order_key(double v) {
  if (v != v) return ~0ull;
  const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);   // (-0 as 0)
  return u >> 63 ? ~u : u | 1ull << 63;
}

__device__ __forceinline__ double of_key(uint64_t k) {
  return __builtin_bit_cast(double, k >> 63 ? k & ~(1ull << 63) : ~k);   // (a NaN's key gives a NaN)
}

// `v` of the lane that the DPP control names, zero where there is none.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t moved(uint64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xf, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xf, false);
  return (uint64_t)hi << 32 | lo;
}

__device__ __forceinline__ uint64_t of_lane(uint64_t v, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
  return (uint64_t)hi << 32 | lo;
}

// The largest key and the sum of a wave, without LDS: rows of 16 lanes by
// shifts of 1, 2, 4 and 8, then the rows' last lanes passed on.
__device__ __forceinline__ uint32_t wave_largest(uint32_t v) {
  const auto take = [&](uint64_t o) { v = (uint32_t)o > v ? (uint32_t)o : v; };
  take(moved<0x111, 0xf>(v));
  take(moved<0x112, 0xf>(v));
  take(moved<0x114, 0xf>(v));
  take(moved<0x118, 0xf>(v));
  take(moved<0x142, 0xa>(v));
  take(moved<0x143, 0xc>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// (the high halves, and the low ones where more than one lane has the highest)
__device__ __forceinline__ uint64_t wave_largest(uint64_t v) {
  const uint32_t hi = wave_largest((uint32_t)(v >> 32));
  const uint64_t have = __ballot((uint32_t)(v >> 32) == hi);
  if ((have & (have - 1)) == 0) return of_lane(v, __builtin_ctzll(have));
  return (uint64_t)hi << 32 | wave_largest((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
}

__device__ __forceinline__ double wave_sum(double v) {
  const auto add = [&](uint64_t o) { v += __builtin_bit_cast(double, o); };
  add(moved<0x111, 0xf>(__builtin_bit_cast(uint64_t, v)));
  add(moved<0x112, 0xf>(__builtin_bit_cast(uint64_t, v)));
  add(moved<0x114, 0xf>(__builtin_bit_cast(uint64_t, v)));
  add(moved<0x118, 0xf>(__builtin_bit_cast(uint64_t, v)));
  add(moved<0x142, 0xa>(__builtin_bit_cast(uint64_t, v)));
  add(moved<0x143, 0xc>(__builtin_bit_cast(uint64_t, v)));
  return __builtin_bit_cast(double, of_lane(__builtin_bit_cast(uint64_t, v), 63));
}

// A wave's view of one token: expert lane + 64 j in its slot j.
template <int J>
__device__ __forceinline__ void load_logits(const Route& p, int64_t t, double (&l)[J], float (&bias)[J]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = lane + 64 * j, at = e < p.n_experts ? e : p.n_experts - 1;
    bias[j] = p.bias ? p.bias[at] : 0.0f;
    double part[R_SPLITS];
#pragma unroll
    for (int s = 0; s < R_SPLITS; ++s) part[s] = s < p.splits ? __builtin_nontemporal_load(p.logits + ((int64_t)s * p.n_tok + t) * p.n_experts + at) : 0.0;
    l[j] = part[0];
#pragma unroll
    for (int s = 1; s < R_SPLITS; ++s) l[j] += part[s];
  }
}

// Scores in the place of logits.
template <int J>
__device__ __forceinline__ void make_scores(const Route& p, double (&v)[J]) {
  const int lane = threadIdx.x & 63;
  if (p.score == QR_SCORE_SIGMOID) {
#pragma unroll
    for (int j = 0; j < J; ++j) v[j] = 1.0 / (1.0 + exp(-v[j]));
    return;
  }
  uint64_t top = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const uint64_t k = order_key(v[j]);
    if (lane + 64 * j < p.n_experts && k > top) top = k;
  }
  const double most = of_key(wave_largest(top));
  double sum = 0.0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    v[j] = exp(v[j] - most);
    if (lane + 64 * j < p.n_experts) sum += v[j];
  }
  sum = wave_sum(sum);
#pragma unroll
  for (int j = 0; j < J; ++j) v[j] /= sum;
}

// The top_k largest of v + bias, largest first: round r's into lane r, with its v
// and the key it was found by; with NEXT `next`, of the round behind it (0: there
// is none). Among equals the lowest.
struct Found {
  int expert;
  double value;
  uint64_t key, next;
};

template <int J, bool NEXT>
__device__ __forceinline__ Found find_largest(const Route& p, const double (&v)[J], const float (&bias)[J]) {
  const int lane = threadIdx.x & 63;
  uint64_t key[J];
#pragma unroll
  for (int j = 0; j < J; ++j)
    key[j] = lane + 64 * j < p.n_experts && bias[j] != -__builtin_inff() ? order_key(v[j] + (double)bias[j]) : 0;
  Found f = {-1, 0.0, 0, 0};
  const int rounds = NEXT ? p.top_k + 1 : p.top_k;
  // up to four to a lane are sorted there first (equal ones stay in their order),
  // and a round then looks at the lanes' first ones only: one token's choice of 8
  // out of 256 5.4 us, 6.1 without
  if constexpr (J <= 4) {
    int expert[J];
#pragma unroll
    for (int j = 0; j < J; ++j) expert[j] = lane + 64 * j;
#pragma unroll
    for (int n = J - 1; n > 0; --n)
#pragma unroll
      for (int j = 0; j < n; ++j) {
        const bool swap = key[j + 1] > key[j];
        const uint64_t k = key[j];
        const int e = expert[j];
        key[j] = swap ? key[j + 1] : k;
        key[j + 1] = swap ? k : key[j + 1];
        expert[j] = swap ? expert[j + 1] : e;
        expert[j + 1] = swap ? e : expert[j + 1];
      }
    for (int r = 0; r < rounds; ++r) {
      const uint64_t best = wave_largest(key[0]);
      if (lane == r - 1) f.next = best;
      if (best == 0 || r == p.top_k) break;
      const uint64_t have = __ballot(key[0] == best);
      int from = __builtin_ctzll(have);
      if (have & (have - 1)) from = (int)(~wave_largest(key[0] == best ? ~(uint32_t)expert[0] : 0u) & 63u);
      const int at = __builtin_amdgcn_readlane(expert[0], from);
      if (lane == from) {
#pragma unroll
        for (int j = 0; j < J - 1; ++j) {
          key[j] = key[j + 1];
          expert[j] = expert[j + 1];
        }
        key[J - 1] = 0;
      }
      if (lane == r) {
        f.expert = at;
        f.key = best;
      }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const double o = __shfl(v[j], f.expert & 63);
      if (f.expert >> 6 == j) f.value = o;   // (-1: none)
    }
    return f;
  }
  for (int r = 0; r < rounds; ++r) {
    uint64_t best = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) best = key[j] > best ? key[j] : best;
    best = wave_largest(best);
    if (lane == r - 1) f.next = best;
    if (best == 0 || r == p.top_k) break;
    // the first slot that has one, its first lane
    int at = -1;
    double won = 0.0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const uint64_t have = __ballot(key[j] == best);
      if (at >= 0 || have == 0) continue;
      const int from = __builtin_ctzll(have);
      at = 64 * j + from;
      won = __builtin_bit_cast(double, of_lane(__builtin_bit_cast(uint64_t, v[j]), from));
      if (lane == from) key[j] = 0;
    }
    if (lane == r) {
      f.expert = at;
      f.value = won;
      f.key = best;
    }
  }
  return f;
}

__device__ __forceinline__ void store_choice(const Route& p, int64_t t, const Found& f) {
  const int lane = threadIdx.x & 63;
  double w = f.value;
  if (p.renorm) {
    const double sum = wave_sum(w);
    w = sum == 0.0 ? 0.0 : w / sum;
  }
  if (lane < p.top_k) {
    p.ids[t * p.top_k + lane] = f.expert;
    p.weights[t * p.top_k + lane] = f.expert < 0 ? 0.0f : (float)(w * (double)p.factor);
  }
}

// One wave per token. Rounds of the largest key by DPP (through LDS permutes one
// token took 23 us); 5.4 us for one token of 256 experts, some 6 for 2048.
template <int J>
__global__ __launch_bounds__(256) void k_route_choose(Route p) {
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= p.n_tok) return;
  double v[J];
  float bias[J];
  load_logits<J>(p, t, v, bias);
  make_scores<J>(p, v);
  store_choice(p, t, find_largest<J, false>(p, v, bias));
}

// All of one token of a small router: a wave takes every WAVES-th expert's logit,
// the first one makes the choice. One launch instead of two, and none of the
// matrix instructions' 15 rows in 16 that a single token leaves empty; 5 us, the
// time of its dependent steps.
constexpr int SMALL_WAVES = 8, SMALL_EXPERTS = 16;

template <int SRC, int WSRC>
__global__ __launch_bounds__(SMALL_WAVES* WAVE) void k_route_small(Route p) {
  __shared__ double logits[SMALL_EXPERTS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.x;
  const uint8_t* x = reinterpret_cast<const uint8_t*>(p.x) + t * p.x_stride * (SRC == QR_BF16 ? 2 : 4);
  const int whole = p.n_in / (8 * WAVE) * (8 * WAVE);
  for (int e = wave; e < p.n_experts; e += SMALL_WAVES) {
    const uint8_t* w = reinterpret_cast<const uint8_t*>(p.w) + (int64_t)e * p.n_in * (WSRC == QR_BF16 ? 2 : 4);
    double sum = 0.0;
#pragma unroll 4
    for (int at = 8 * lane; at < whole; at += 8 * WAVE) {
      const Eight<SRC> a = eight_at<SRC>(x, at);
      const Eight<WSRC> b = eight_at<WSRC>(w, at);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = __builtin_fma(a.get(i), b.get(i), sum);
    }
    if (whole < p.n_in) {
      float a[8], b[8];
      load8<SRC>(x, whole + 8 * lane, p.n_in, a);
      load8<WSRC>(w, whole + 8 * lane, p.n_in, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)a[i], (double)b[i], sum);
    }
    sum = wave_sum(sum);
    if (lane == 0) logits[e] = sum;
  }
  __syncthreads();
  if (wave != 0) return;
  const int at = lane < p.n_experts ? lane : p.n_experts - 1;
  double v[1] = {logits[at]};
  const float bias[1] = {p.bias ? p.bias[at] : 0.0f};
  make_scores<1>(p, v);
  store_choice(p, t, find_largest<1, false>(p, v, bias));
}

// Rough logits of many tokens, both sides bf16: the bf16 matrix cores' fp32 sums
// of ROUGH_SUM products, added up in 64 bits. k_route_settle takes exact ones
// where they matter. 2048 tokens, 256 experts, 7168 values: 27 us, of which the
// products are 6; the steps' parts follow each other in the one workgroup of a CU
// (two of them, or loads five steps ahead: no faster).
//
// 64 experts x 128 tokens per workgroup, 64 values of the sum per step through
// LDS, loads ROUGH_AHEAD steps ahead. In LDS the 16-byte piece c of row r lies at
// r * 128 + (c ^ (r / 2 % 8)) * 16: sixteen lanes that take one piece of
// neighbouring rows meet all banks.
constexpr int ROUGH_SUM = 128, ROUGH_E = 64, ROUGH_T = 128, ROUGH_K = 64, ROUGH_AHEAD = 3;

__global__ __launch_bounds__(512) void k_route_rough(Route p, int expert_tiles, int token_tiles) {
  __shared__ u32x4 tile[2][(ROUGH_E + ROUGH_T) * 8];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lk = lane >> 4;
  // workgroups are dealt to the 8 dies in turn: each die gets neighbouring tiles,
  // so that the experts' tiles of one token tile find it in one L2
  const int all = (int)gridDim.x, die = (int)(blockIdx.x % 8);
  int block = die * (all / 8) + (die < all % 8 ? die : all % 8) + (int)(blockIdx.x / 8);
  const int be = block % expert_tiles;
  block /= expert_tiles;
  const int bt = block % token_tiles, split = block / token_tiles;
  // staging: piece tid % 8 of rows tid / 8 (experts) and 64 and 128 behind it (tokens)
  const int row = tid >> 3, col = tid & 7;
  const uint16_t* src[3];
  {
    const int e = be * ROUGH_E + row, t = bt * ROUGH_T + row;
    src[0] = reinterpret_cast<const uint16_t*>(p.w) + (int64_t)(e < p.n_experts ? e : p.n_experts - 1) * p.n_in + 8 * col;
    src[1] = reinterpret_cast<const uint16_t*>(p.x) + (int64_t)(t < p.n_tok ? t : p.n_tok - 1) * p.x_stride + 8 * col;
    src[2] = reinterpret_cast<const uint16_t*>(p.x) + (int64_t)(t + 64 < p.n_tok ? t + 64 : p.n_tok - 1) * p.x_stride + 8 * col;
  }
  const int put = row * 8 + (col ^ ((row >> 1) & 7));
  u32x4 raw[ROUGH_AHEAD][3];
  auto load = [&](u32x4 (&r)[3], int step) {
#pragma unroll
    for (int i = 0; i < 3; ++i) r[i] = __builtin_bit_cast(u32x4, *reinterpret_cast<const u16x8_any*>(src[i] + step * ROUGH_K));
  };
  float sq[3] = {};
  auto stage = [&](const u32x4 (&r)[3], u32x4* to) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      to[put + i * 64 * 8] = r[i];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bf16x2 two = __builtin_bit_cast(bf16x2, (uint32_t)r[i][k]);
        sq[i] = __builtin_amdgcn_fdot2_f32_bf16(two, two, sq[i], false);
      }
    }
  };
  // a wave's part of the tile: 32 experts x 32 tokens
  const int we = (wave & 1) * 32, wt = ROUGH_E + (wave >> 1) * 32;
  f64x4 acc[2][2] = {};
  f32x4 sum[2][2] = {};
  auto multiply = [&](const u32x4* from) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      bf16x8 a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int ra = we + 16 * i + li, rb = wt + 16 * i + li;
        a[i] = __builtin_bit_cast(bf16x8, from[ra * 8 + ((4 * k + lk) ^ ((ra >> 1) & 7))]);
        b[i] = __builtin_bit_cast(bf16x8, from[rb * 8 + ((4 * k + lk) ^ ((rb >> 1) & 7))]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) sum[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], sum[i][j], 0, 0, 0);
    }
  };
  auto flush = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][j][v] += (double)sum[i][j][v];
        sum[i][j] = f32x4{0, 0, 0, 0};
      }
  };
  // whole steps; what is left of the rows is the last split's, behind them
  const int steps = p.n_in / ROUGH_K;
  const int from = (int)((int64_t)steps * split / p.splits), to = (int)((int64_t)steps * (split + 1) / p.splits);
#pragma unroll
  for (int s = 0; s < ROUGH_AHEAD; ++s)
    if (from + s < to) load(raw[s], from + s);
  if (from < to) stage(raw[0], tile[0]);
  if (from + ROUGH_AHEAD < to) load(raw[0], from + ROUGH_AHEAD);
  __syncthreads();
  int s = from;
  // (no conditions here: where loads may or may not be on their way, all are waited for)
  for (; s + 2 * ROUGH_AHEAD < to; s += ROUGH_AHEAD) {
#pragma unroll
    for (int u = 0; u < ROUGH_AHEAD; ++u) {
      const int now = (s + u - from) & 1;
      stage(raw[(u + 1) % ROUGH_AHEAD], tile[now ^ 1]);
      load(raw[(u + 1) % ROUGH_AHEAD], s + u + 1 + ROUGH_AHEAD);
      multiply(tile[now]);
      if (now) flush();
      __syncthreads();
    }
  }
  for (; s < to; s += ROUGH_AHEAD) {
#pragma unroll
    for (int u = 0; u < ROUGH_AHEAD; ++u) {
      const int now = (s + u - from) & 1;
      if (s + u >= to) break;
      if (s + u + 1 < to) {
        stage(raw[(u + 1) % ROUGH_AHEAD], tile[now ^ 1]);
        if (s + u + 1 + ROUGH_AHEAD < to) load(raw[(u + 1) % ROUGH_AHEAD], s + u + 1 + ROUGH_AHEAD);
      }
      multiply(tile[now]);
      if (now) flush();
      __syncthreads();
    }
  }
  flush();
  if (split == p.splits - 1 && p.n_in % ROUGH_K != 0) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      u16x8_any v;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = steps * ROUGH_K + 8 * col + k < p.n_in ? src[i][steps * ROUGH_K + k] : (uint16_t)0;
      raw[0][i] = __builtin_bit_cast(u32x4, v);
    }
    stage(raw[0], tile[0]);
    __syncthreads();
    multiply(tile[0]);
    flush();
  }
  // a lane holds experts 4 lk + v of a tile for token li
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int t = bt * ROUGH_T + wt - ROUGH_E + 16 * j + li;
    if (t >= p.n_tok) continue;
    double* out = p.logits + ((int64_t)split * p.n_tok + t) * p.n_experts;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int e = be * ROUGH_E + we + 16 * i + 4 * lk + v;
        if (e < p.n_experts) out[e] = acc[i][j][v];
      }
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) {
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) sq[i] += __shfl_xor(sq[i], d);
    const int e = be * ROUGH_E + row, t = bt * ROUGH_T + row + 64 * (i - 1);
    if (col != 0) continue;
    if (i == 0 && bt == 0 && e < p.n_experts) p.squares[(int64_t)p.splits * p.n_tok + (int64_t)split * p.n_experts + e] = sq[i];
    if (i > 0 && be == 0 && t < p.n_tok) p.squares[(int64_t)split * p.n_tok + t] = sq[i];
  }
}

// How far a token's rough logits may be off: fp32 sums of ROUGH_SUM exact
// products, each addition off by a last place of the products' magnitudes added
// up (twice what rounding does), and those at most the rows' lengths multiplied.
// Zero for a row of zeros, whose logits are exact, unless a weight may be no
// number: the choice that stands by itself then takes zeros for its logits. (By
// one wave.)
__device__ __forceinline__ double rough_error(const Route& p, int64_t t) {
  const int lane = threadIdx.x & 63;
  float x = 0.0f, w = 0.0f;
  for (int s = 0; s < p.splits; ++s) x += p.squares[(int64_t)s * p.n_tok + t];
  for (int e = lane; e < p.n_experts; e += WAVE) {
    float v = 0.0f;
    for (int s = 0; s < p.splits; ++s) v += p.squares[(int64_t)p.splits * p.n_tok + (int64_t)s * p.n_experts + e];
    w = v > w || v != v ? v : w;
  }
  const double most = of_key(wave_largest(order_key((double)w)));
  if (x < 0x1p-80f) {            // squares and products may have vanished
    uint32_t any = 0;
    const uint16_t* row = reinterpret_cast<const uint16_t*>(p.x) + t * p.x_stride;
    for (int at = lane; at < p.n_in; at += WAVE) any |= row[at] & 0x7fffu;
    return __ballot(any != 0) || !(most < __builtin_inf()) ? __builtin_inf() : 0.0;
  }
  if (most < 0x1p-80) return __builtin_inf();
  return ROUGH_SUM * 0x1p-23 * 1.02 * __builtin_sqrt((double)x) * __builtin_sqrt(most);
}

// The exact logits of N experts of a list, by one wave.
template <int N>
__device__ __forceinline__ void exact_logits(const Route& p, int64_t t, const uint16_t* list, double* out) {
  const int lane = threadIdx.x & 63;
  const uint16_t* x = reinterpret_cast<const uint16_t*>(p.x) + t * p.x_stride;
  const uint16_t* w[N];
#pragma unroll
  for (int q = 0; q < N; ++q)
    w[q] = reinterpret_cast<const uint16_t*>(p.w) + (int64_t)__builtin_amdgcn_readfirstlane(list[q]) * p.n_in;
  double sum[N] = {};
  const int whole = p.n_in / (8 * WAVE) * (8 * WAVE);
#pragma unroll 2
  for (int at = 8 * lane; at < whole; at += 8 * WAVE) {
    const u16x8_any a = __builtin_nontemporal_load(reinterpret_cast<const u16x8_any*>(x + at));
    u16x8_any b[N];
#pragma unroll
    for (int q = 0; q < N; ++q) b[q] = *reinterpret_cast<const u16x8_any*>(w[q] + at);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double v = (double)bf16_value(a[i]);
#pragma unroll
      for (int q = 0; q < N; ++q) sum[q] = __builtin_fma(v, (double)bf16_value(b[q][i]), sum[q]);
    }
  }
  if (whole < p.n_in) {
    float a[8], b[8];
    load8<QR_BF16>(x, whole + 8 * lane, p.n_in, a);
#pragma unroll
    for (int q = 0; q < N; ++q) {
      load8<QR_BF16>(w[q], whole + 8 * lane, p.n_in, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[q] = __builtin_fma((double)a[i], (double)b[i], sum[q]);
    }
  }
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const double l = wave_sum(sum[q]);
    if (lane == 0) out[q] = l;
  }
}

// The choice from rough logits, off by up to d: one workgroup per token. What is
// found as the largest, u = logit or (with a bias, of sigmoids, whose slope is at
// most 1/4) score + bias, is off by up to d or d / 4. The chosen ones get exact
// logits, for their weights, and so does all that lies so near to one that it may
// come before it; the choice is then made again, of the scores, which is the one
// that exact logits throughout would give. Near is also what the 64 bits of a score
// (+ bias) may not tell apart: that part of the margin is seen only where sigmoids
// near one, scores of no size or a huge bias round the differences away. Of two
// logits found more than 2 d apart that both give scores of zero (below -709 of
// themselves, or of the largest), the lower one is found below -690.
//
// 2048 tokens, 8 of 256 experts: 41 us, some 30 of them for nine exact logits a
// token. Vector instructions are issued in 56% of the time, four for each product
// of a sum (conversions to 64 bits most of them) and half as many again for the
// choice; a sum's halves or quarters dealt to the waves: no faster. 64 registers,
// for eight workgroups to a CU, which hide each other's waits (100: 55 us); 9 more,
// of the choice's state, lie in scratch memory during the sums (13 where there are
// 512 experts, 23 with 1024).
template <int J>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(J <= 4 ? 8 : J == 8 ? 4 : 2))) void k_route_settle(Route p) {
  __shared__ double exact[64 * J];
  __shared__ uint16_t list[64 * J];
  __shared__ int listed;
  __shared__ double rough;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.x;
  double l[J];
  float bias[J];
  int at[J];                     // where the list has this lane's experts, or -1
  double u[J];
  Found f;
  uint64_t unsure = 0;
  if (wave == 0) {
    load_logits<J>(p, t, l, bias);
#pragma unroll
    for (int j = 0; j < J; ++j) u[j] = p.bias ? 1.0 / (1.0 + exp(-l[j])) : l[j];
    f = find_largest<J, true>(p, u, bias);
  } else if (wave == 1) {
    const double d = rough_error(p, t);
    if (lane == 0) rough = d;
  }
  __syncthreads();
  if (wave == 0) {
    const double d = rough;
    const double u0 = of_key(f.key), u1 = of_key(f.next);
    double margin;
    if (p.bias) margin = 0.52 * d + 0x1p-50 * (1.0 + __builtin_fabs(u0) + __builtin_fabs(u1));
    else if (p.score == QR_SCORE_SIGMOID) margin = u1 < -690.0 ? __builtin_inf() : 2.0 * d + 0x1p-49 * (1.0 + exp(u0));
    else margin = u1 - of_key(__shfl(f.key, 0)) < -690.0 ? __builtin_inf() : 2.0 * d + 0x1p-48;
    const uint64_t found = __ballot(f.expert >= 0);
    unsure = __ballot(f.expert >= 0 && f.next != 0 && !(u0 - u1 > margin));
    if (unsure == 0) {           // the choice stands as it is
      if (f.expert >= 0) list[lane] = (uint16_t)f.expert;
      if (lane == 0) listed = d == 0.0 ? 0 : __builtin_popcountll(found);
    } else {
      uint32_t want = 0;         // of this lane's experts: bit j
      for (uint64_t left = unsure; left; left &= left - 1) {
        const int r = __builtin_ctzll(left);
        const double upper = __shfl(u0 + margin, r), lower = __shfl(u1 - margin, r);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const double v = u[j] + (double)bias[j];
          if (lane + 64 * j < p.n_experts && !(v > upper) && !(v < lower)) want |= 1u << j;
        }
      }
      for (int r = 0; r < p.top_k; ++r) {
        const int e = __builtin_amdgcn_readlane(f.expert, r);
        if (e >= 0 && lane == (e & 63)) want |= 1u << (e >> 6);
      }
      if (d == 0.0) want = 0;
      int n = 0;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const bool is = want >> j & 1;
        const uint64_t all = __ballot(is);
        at[j] = is ? n + __builtin_popcountll(all & ((1ull << lane) - 1)) : -1;
        if (is) list[at[j]] = (uint16_t)(lane + 64 * j);
        n += __builtin_popcountll(all);
      }
      if (lane == 0) listed = n;
    }
  }
  __syncthreads();
  const int n = __builtin_amdgcn_readfirstlane(listed);
  // dealt evenly: a wave's experts share the token's row
  for (int i = n * wave / 4; i < n * (wave + 1) / 4; i += 2) {
    if (n * (wave + 1) / 4 - i == 1) exact_logits<1>(p, t, list + i, exact + i);
    else exact_logits<2>(p, t, list + i, exact + i);
  }
  __syncthreads();
  if (wave != 0) return;
  if (unsure == 0) {
    // the first one is the largest; a softmax is divided by the chosen ones' sum
    const double v = n ? exact[f.expert >= 0 ? lane : 0] : 0.0, most = __shfl(v, 0);
    f.value = f.expert < 0 ? 0.0 : p.score == QR_SCORE_SIGMOID ? 1.0 / (1.0 + exp(-v)) : exp(v - most);
    store_choice(p, t, f);
    return;
  }
#pragma unroll
  for (int j = 0; j < J; ++j)
    if (at[j] >= 0) l[j] = exact[at[j]];
  make_scores<J>(p, l);
  store_choice(p, t, find_largest<J, false>(p, l, bias));
}

// ---------------------------------------------------------------------------
// the experts

struct Moe {
  const int8_t *gate, *up, *down;
  const float *gated, *upd, *downd;
  const int8_t* x;
  const float* xd;
  const int32_t* ids;
  const float* weights;
  int8_t* h;             // [pairs][64 * blocks] hidden codes
  float* hd;             // [pairs][scale_pitch] their scales
  const void* residual;
  void* y;
  int64_t expert_rows, residual_stride, y_stride;
  int n_experts, n_in, n_mid, in_bytes, mid_bytes, blocks, scale_pitch, n_tok, top_k, act;
};

constexpr int M_WAVES = 8;
constexpr int M_BLOCK = 64;            // hidden channels of one scale
constexpr int NO_EXPERT = 0xffff;
constexpr int MASK_WORDS = QR_MOE_MAX_EXPERTS / 32;

// The pairs (a token and a slot) of a run that meet one expert.
struct Met {
  int expert;            // -1: none
  int n;
  uint64_t set;          // up to 64 pairs: which they are
  const uint16_t* list;  // more: their numbers
};

// Up to 64 pairs: a wave holds a choice per lane, finds the rank-th expert (in
// the order in which they first appear) and its pairs with ballots alone.
__device__ __forceinline__ int choice_of(const Moe& m, int first, int n) {
  const int lane = threadIdx.x & 63;
  const int id = lane < n ? m.ids[first + lane] : -1;
  return (uint32_t)id < (uint32_t)m.n_experts ? id : -1;
}

__device__ __forceinline__ Met met_of_few(int choice, int rank) {
  uint64_t left = __ballot(choice >= 0);
  Met r = {-1, 0, 0, nullptr};
  for (; left; --rank) {
    const int e = __builtin_amdgcn_readlane(choice, __builtin_ctzll(left));
    const uint64_t set = __ballot(choice == e);
    if (rank == 0) {
      r.expert = e;
      r.n = __builtin_popcountll(set);
      r.set = set;
      break;
    }
    left &= ~set;
  }
  return r;
}

// The rank-th expert of a set in LDS, or -1.
__device__ __forceinline__ int expert_of_rank(const uint32_t* mask, int rank) {
  int e = -1;
#pragma unroll 8
  for (int w = 0; w < MASK_WORDS; ++w) {
    uint32_t bits = mask[w];
    const int n = __builtin_popcount(bits);
    if (rank >= 0 && rank < n) {
      for (int i = 0; i < rank; ++i) bits &= bits - 1;
      e = 32 * w + __builtin_ctz(bits);
    }
    rank -= n;
  }
  return e;
}

// The choices of n pairs into LDS, and the set of experts that they meet.
__device__ __forceinline__ void read_choices(const Moe& m, int first, int n, uint16_t* ids, uint32_t* mask) {
  for (int i = threadIdx.x; i < MASK_WORDS; i += M_WAVES * WAVE) mask[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += M_WAVES * WAVE) {
    const int id = m.ids[first + i];
    const bool is = (uint32_t)id < (uint32_t)m.n_experts;
    ids[i] = (uint16_t)(is ? id : NO_EXPERT);
    if (is) atomicOr(&mask[id >> 5], 1u << (id & 31));
  }
  __syncthreads();
}

// The at-th of the expert's pairs, the last one again behind them.
template <bool FEW>
__device__ __forceinline__ int pair_of(const Met& r, int at) {
  if (at > r.n - 1) at = r.n - 1;
  if (!FEW) return r.list[at];
  // the at-th set bit, halving the words that it may lie in
  uint32_t word = (uint32_t)r.set;
  int found = 0, below = __builtin_popcount(word);
  if (at >= below) {
    at -= below;
    word = (uint32_t)(r.set >> 32);
    found = 32;
  }
#pragma unroll
  for (int width = 16; width > 0; width >>= 1) {
    below = __builtin_popcount(word & ((1u << width) - 1));
    if (at >= below) {
      at -= below;
      word >>= width;
      found += width;
    }
  }
  return found;
}

constexpr int HIDDEN_TILES = 4;        // of 16 pairs, whose products share the weights they are made with

// Gate and up products of one block of 64 hidden channels for 16 TT pairs of
// one expert, and their 8-bit hidden values. Waves 0-3 have 16 channels each and
// the first half of the sum, waves 4-7 the second: a wave reads neighbouring
// lines of 32 rows, four stages of 4 KB ahead.
template <int TT, bool FEW>
__device__ __forceinline__ void hidden_block(const Moe& m, const Met& met, int first, int block,
                                             i32x4 (*part)[4][2][HIDDEN_TILES][WAVE]) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lk = lane >> 4, group = wave & 3, half = wave >> 2;
  const int c0 = M_BLOCK * block + 16 * group;
  const int64_t rows = (int64_t)__builtin_amdgcn_readfirstlane(met.expert) * m.expert_rows;
  const int first_row = c0 < m.n_mid ? c0 : m.n_mid - 1, row_left = m.n_mid - 1 - first_row < 15 ? m.n_mid - 1 - first_row : 15;
  const Buffer gate = buffer_of(m.gate + (rows + first_row) * m.in_bytes, (uint32_t)(row_left + 1) * (uint32_t)m.in_bytes);
  const Buffer up = buffer_of(m.up + (rows + first_row) * m.in_bytes, (uint32_t)(row_left + 1) * (uint32_t)m.in_bytes);
  const Buffer xs = buffer_of(m.x, (uint32_t)m.n_tok * (uint32_t)m.in_bytes);
  uint32_t at[2], x[TT];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = 8 * h + (li & 7);        // rows behind the last repeat it
    at[h] = (uint32_t)(r < row_left ? r : row_left) * (uint32_t)m.in_bytes + 64 * (li >> 3) + 16 * lk;
  }
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int i = first + 16 * j + li;
    x[j] = i < met.n ? (uint32_t)(pair_of<FEW>(met, i) / m.top_k) * (uint32_t)m.in_bytes + 16 * lk : NOWHERE;
  }
  // what the epilogue needs: two channels of one pair per lane
  const int hc = M_BLOCK * block + 2 * (lane & 31);
  float gd[2], ud[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int64_t r = rows + (hc + e < m.n_mid ? hc + e : m.n_mid - 1);
    gd[e] = m.gated[r];
    ud[e] = m.upd[r];
  }
  const int chunks = m.in_bytes / 128, middle = (chunks + 1) / 2;
  const int from = half ? middle : 0, to = half ? chunks : middle;
  i32x4 acc[2][TT] = {};
  struct Stage {
    i32x4 a[2][2], b[2][TT];
  };
  pipeline<TT == 1 ? 4 : 2, Stage>(from, to, 1,
      [&](Stage& s, int k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          s.a[0][h] = load16_once(gate, at[h], k * 128);
          s.a[1][h] = load16_once(up, at[h], k * 128);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < TT; ++j) s.b[h][j] = load16(xs, x[j], k * 128 + 64 * h);
      },
      [&](Stage& s, int) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          turn(s.a[g][0], s.a[g][1]);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < TT; ++j)
              acc[g][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(s.a[g][h], s.b[h][j], acc[g][j], 0, 0, 0);
        }
      });
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int j = 0; j < TT; ++j) part[half][group][g][j][lane] = acc[g][j];
  __syncthreads();
  // half a wave per pair
#pragma unroll 1
  for (int q = 2 * wave + (lane >> 5); q < 16 * TT; q += 2 * M_WAVES) {
    if (first + q >= met.n) break;
    const int pair = pair_of<FEW>(met, first + q), c = 2 * (lane & 31);
    const TokenScale d = token_scale(m.xd[pair / m.top_k]);
    const int* sums = reinterpret_cast<const int*>(part);
    float v[2];
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      // sum of channel 16 g' + 4 lk + i of column li: element i of lane 16 lk + li
      const int of = (((c >> 4) * 2 * HIDDEN_TILES + (q >> 4)) * WAVE + ((c >> 2) & 3) * 16 + (q & 15)) * 4 + (c & 3) + e;
      constexpr int UP = HIDDEN_TILES * WAVE * 4, HALF = 4 * 2 * HIDDEN_TILES * WAVE * 4;
      // in 64 bits, so that the codes that are made of it do not hang on the
      // last place of an exp
      const double g = (double)scaled(sums[of] + sums[of + HALF], d, gd[e], 0.0f);
      const double u = (double)scaled(sums[of + UP] + sums[of + UP + HALF], d, ud[e], 0.0f);
      v[e] = hc + e < m.n_mid ? (float)(activation(m.act, g) * u) : 0.0f;
      const uint32_t mag = __builtin_bit_cast(uint32_t, v[e]) & 0x7fffffffu;
      top = mag > top ? mag : top;
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
      const uint32_t o = (uint32_t)__shfl_xor((int)top, s);
      top = o > top ? o : top;
    }
    const CodeScale s = code_scale(top);
    const int lo = s.finite ? (int)__builtin_rintf(v[0] * s.inv) : 0, hi = s.finite ? (int)__builtin_rintf(v[1] * s.inv) : 0;
    *reinterpret_cast<uint16_t*>(m.h + ((int64_t)pair * m.blocks + block) * M_BLOCK + c) =
        (uint16_t)((lo & 0xff) | (hi & 0xff) << 8);
    if ((lane & 31) == 0) m.hd[(int64_t)pair * m.scale_pitch + block] = s.d;
  }
  __syncthreads();
}

// One workgroup per expert that is met and block of hidden channels: it finds
// its expert and the expert's pairs in the choices by itself (a captured call
// replays with other choices). FEW: all pairs fit into a wave's lanes.
//
// Bound by the weights' bytes. Eight of 256 experts, 7168 x 2048, for one token:
// 39 us, 6.0 TB/s (merely reading as many bytes from 256 workgroups: 37 us); 113
// of them for 64 tokens: 572 us, 5.8 TB/s. 23 tokens of 8 experts of 4096 x 11008:
// 142 us, 5.1 TB/s, 1376 workgroups being 5.4 rounds of the chip. With 64-bit
// addresses, a batch at a time and through the caches: 54, 748 and 202 us.
template <bool FEW>
__global__ __launch_bounds__(M_WAVES* WAVE) void k_moe_hidden(Moe m) {
  extern __shared__ uint16_t dynamic[];
  __shared__ uint32_t mask[MASK_WORDS];
  __shared__ int counts[M_WAVES];
  __shared__ i32x4 part[2][4][2][HIDDEN_TILES][WAVE];
  const int pairs = m.n_tok * m.top_k;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int block = (int)(blockIdx.x % (uint32_t)m.blocks), rank = (int)(blockIdx.x / (uint32_t)m.blocks);
  Met met;
  if (FEW) {
    met = met_of_few(choice_of(m, 0, pairs), rank);
    if (met.expert < 0) return;
  } else {
    uint16_t *ids = dynamic, *list = dynamic + pairs;
    read_choices(m, 0, pairs, ids, mask);
    met.expert = __builtin_amdgcn_readfirstlane(expert_of_rank(mask, rank));
    if (met.expert < 0) return;
    // its pairs in their order: every wave looks through a run of them
    const int run = ((pairs + M_WAVES - 1) / M_WAVES + 63) & ~63;
    const int from = wave * run, to = from + run < pairs ? from + run : pairs;
    int mine = 0;
    for (int i = from; i < to; i += 64) mine += __builtin_popcountll(__ballot(i + lane < to && ids[i + lane] == met.expert));
    if (lane == 0) counts[wave] = mine;
    __syncthreads();
    int n = 0, put = 0;
#pragma unroll
    for (int w = 0; w < M_WAVES; ++w) {
      put += w < wave ? counts[w] : 0;
      n += counts[w];
    }
    for (int i = from; i < to; i += 64) {
      const bool is = i + lane < to && ids[i + lane] == met.expert;
      const uint64_t all = __ballot(is);
      if (is) list[put + __builtin_popcountll(all & ((1ull << lane) - 1))] = (uint16_t)(i + lane);
      put += __builtin_popcountll(all);
    }
    __syncthreads();
    met.n = __builtin_amdgcn_readfirstlane(n);
    met.list = list;
  }
  for (int at = 0; at < met.n;) {
    const int left = met.n - at;
    if (left <= 16) {
      hidden_block<1, FEW>(m, met, at, block, part);
      at += 16;
    } else if (left <= 32) {
      hidden_block<2, FEW>(m, met, at, block, part);
      at += 32;
    } else {
      hidden_block<4, FEW>(m, met, at, block, part);
      at += 64;
    }
  }
}

constexpr int D_SLOTS = 512;     // partial sums of 16 channels that a workgroup holds

// One expert's sums of 16 output channels over blocks of hidden channels, for
// 16 TT pairs: exact per block, times the block's scale in fp32.
template <int TT, bool FEW>
__device__ __forceinline__ void down_block(const Moe& m, const Met& met, int at, int c0, int from, int to, int first_pair,
                                           float (*sums)[16]) {
  const int lane = threadIdx.x & 63;
  const int li = lane & 15, lk = lane >> 4;
  const int64_t rows = (int64_t)__builtin_amdgcn_readfirstlane(met.expert) * m.n_in;
  const Buffer w = buffer_of(m.down + (rows + c0) * m.mid_bytes,
                             (uint32_t)(m.n_in - c0 < 16 ? m.n_in - c0 : 16) * (uint32_t)m.mid_bytes);
  const uint32_t pairs = (uint32_t)(m.n_tok * m.top_k);
  const Buffer hs = buffer_of(m.h, pairs * (uint32_t)(m.blocks * M_BLOCK)), hds = buffer_of(m.hd, pairs * (uint32_t)(m.scale_pitch * 4));
  uint32_t off[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = 8 * h + (li & 7);        // rows behind the last repeat it
    off[h] = (uint32_t)(c0 + r < m.n_in ? r : m.n_in - 1 - c0) * (uint32_t)m.mid_bytes + 64 * (li >> 3) + 16 * lk;
  }
  int pair[TT];
  uint32_t h[TT], hd[TT];
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    pair[j] = pair_of<FEW>(met, at + 16 * j + li);
    const bool is = at + 16 * j + li < met.n;
    h[j] = is ? (uint32_t)(first_pair + pair[j]) * (uint32_t)(m.blocks * M_BLOCK) + 16 * lk : NOWHERE;
    hd[j] = is ? (uint32_t)(first_pair + pair[j]) * (uint32_t)(m.scale_pitch * 4) : NOWHERE;
  }
  f32x4 acc[TT] = {};
  // four blocks, 256 bytes of a row, at a time; behind the last block the row
  // of codes has zeros up to its next 128, the hidden row nothing
  const int last = m.mid_bytes - 128;
  struct Stage {
    i32x4 a[4], b[4][TT];
    f32x4 d[TT];
  };
  pipeline<2, Stage>(from, to, 4,
      [&](Stage& s, int k) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int c = k * 64 + 128 * u < last ? k * 64 + 128 * u : last;
          s.a[2 * u] = load16_once(w, off[0], c);
          s.a[2 * u + 1] = load16_once(w, off[1], c);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int c = k + u < m.blocks ? k + u : m.blocks - 1;
#pragma unroll
          for (int j = 0; j < TT; ++j) s.b[u][j] = load16(hs, h[j], c * 64);
        }
#pragma unroll
        for (int j = 0; j < TT; ++j) s.d[j] = __builtin_bit_cast(f32x4, load16(hds, hd[j], k * 4));
      },
      [&](Stage& s, int k) {
        turn(s.a[0], s.a[1]);
        turn(s.a[2], s.a[3]);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
          for (int j = 0; j < TT; ++j) {
            const i32x4 p = __builtin_amdgcn_mfma_i32_16x16x64_i8(s.a[u], s.b[u][j], i32x4{0, 0, 0, 0}, 0, 0, 0);
            const float d = k + u < m.blocks ? s.d[j][u] : 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] += d * (float)p[e];
          }
        }
      });
  float wd[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int c = c0 + 4 * lk + e;
    wd[e] = m.downd[rows + (c < m.n_in ? c : m.n_in - 1)];
  }
#pragma unroll
  for (int j = 0; j < TT; ++j)
    if (at + 16 * j + li < met.n) {
      f32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = acc[j][e] * wd[e];
      *reinterpret_cast<f32x4*>(&sums[pair[j]][4 * lk]) = o;
    }
}

template <int DST>
__device__ __forceinline__ float value_at(const void* x, int64_t i) {
  return DST == QR_BF16 ? bf16_value(reinterpret_cast<const uint16_t*>(x)[i]) : reinterpret_cast<const float*>(x)[i];
}

// Up to 512 pairs sorted by expert, in LDS: a thread has a pair, counters of all
// experts give it a place among its expert's (which one does not matter to any
// result) and their running sums the expert's place among those that are met.
struct Sorted {
  uint32_t count[QR_MOE_MAX_EXPERTS];          // pairs, later where an expert's begin
  uint32_t waves[M_WAVES];
  uint16_t experts[D_SLOTS], begin[D_SLOTS + 1], pairs[D_SLOTS];
};

__device__ __forceinline__ int sort_pairs(const Moe& m, int first, int n, Sorted& s, uint16_t* ids) {
  constexpr int EACH = QR_MOE_MAX_EXPERTS / (M_WAVES * WAVE);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int id = tid < n ? m.ids[first + tid] : -1;
  const bool is = (uint32_t)id < (uint32_t)m.n_experts;
  if (tid < n) ids[tid] = (uint16_t)(is ? id : NO_EXPERT);
#pragma unroll
  for (int i = 0; i < EACH; ++i) s.count[EACH * tid + i] = 0;
  __syncthreads();
  uint32_t place = 0;
  if (is) place = atomicAdd(&s.count[id], 1u);
  __syncthreads();
  // running sums of pairs (low half) and of experts that have any (high half)
  uint32_t mine[EACH], sum = 0;
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    mine[i] = s.count[EACH * tid + i];
    sum += mine[i] ? mine[i] + 0x10000u : 0u;
  }
  uint32_t up = sum;
#pragma unroll
  for (int d = 1; d < WAVE; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_up((int)up, d);
    if (lane >= d) up += o;
  }
  if (lane == 63) s.waves[wave] = up;
  __syncthreads();
  uint32_t before = up - sum, all = 0;
#pragma unroll
  for (int w = 0; w < M_WAVES; ++w) {
    if (w < wave) before += s.waves[w];
    all += s.waves[w];
  }
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    if (!mine[i]) continue;
    s.experts[before >> 16] = (uint16_t)(EACH * tid + i);
    s.begin[before >> 16] = (uint16_t)before;
    s.count[EACH * tid + i] = before & 0xffffu;
    before += mine[i] + 0x10000u;
  }
  if (tid == 0) s.begin[all >> 16] = (uint16_t)all;
  __syncthreads();
  if (is) s.pairs[s.count[id] + place] = (uint16_t)tid;
  __syncthreads();
  return __builtin_amdgcn_readfirstlane((int)(all >> 16));
}

// 16 output channels of a run of tokens per workgroup. Its waves take the
// experts that these tokens meet in turn (with fewer than eight of them, parts
// of an expert's sum), every pair's sums go to LDS, and a token's are added up
// in the order of its slots.
//
// Bound by the weights' bytes, and by the start of every expert's: eight experts
// of 2048 x 7168 for one token 24.5 us, 4.8 TB/s (merely read: 21 us), 113 for 64
// tokens 320 us, 5.2 TB/s, 8 of 11008 x 4096 for 23 tokens 77 us (merely read: 69
// to 75). Two workgroups to a CU, within 128 registers; loads that run on into
// the wave's next expert spilled 40 of them (555 us). Every run of tokens reads the
// rows of the experts that it meets for itself: 64, 128, 256 and 1024 tokens, 8 of
// 256 experts (226 to 256 met) 586, 1158, 1973 and 7874 us, 3.3, 6.7, 13 and 52 GB
// from memory.
template <int DST, int MOST, bool FEW>
__global__ __launch_bounds__(M_WAVES* WAVE) __attribute__((amdgpu_waves_per_eu(MOST == 1 ? 4 : 2))) void k_moe_down(Moe m, int tokens_each) {
  constexpr int PAIRS = FEW ? 64 : D_SLOTS;
  struct None {};
  __shared__ std::conditional_t<FEW, None, Sorted> sorted;
  __shared__ uint16_t ids[PAIRS];
  __shared__ float weights[PAIRS];
  __shared__ float sums[D_SLOTS][16];
  const int tiles = (m.n_in + 15) / 16;
  const int c0 = (int)(blockIdx.x % (uint32_t)tiles) * 16, t0 = (int)(blockIdx.x / (uint32_t)tiles) * tokens_each;
  const int tokens = m.n_tok - t0 < tokens_each ? m.n_tok - t0 : tokens_each;
  const int first = t0 * m.top_k, pairs = tokens * m.top_k;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (tid < pairs) weights[tid] = m.weights[first + tid];
  int choice = -1, met_all = 0;
  if constexpr (FEW) {
    choice = choice_of(m, first, pairs);
    if (tid < pairs) ids[tid] = (uint16_t)(choice < 0 ? NO_EXPERT : choice);
    for (uint64_t left = __ballot(choice >= 0); left; ++met_all)
      left &= ~__ballot(choice == __builtin_amdgcn_readlane(choice, __builtin_ctzll(left)));
  } else {
    met_all = sort_pairs(m, first, pairs, sorted, ids);
  }
  // parts of a sum in groups of four blocks
  const int groups = m.scale_pitch / 4;
  int parts = 1;
  if (met_all > 0 && met_all < M_WAVES) {
    parts = M_WAVES / met_all;
    if (parts > D_SLOTS / pairs) parts = D_SLOTS / pairs;
    if (parts > groups) parts = groups;
  }
  for (int item = wave; item < met_all * parts; item += M_WAVES) {
    const int part = item % parts;
    Met met;
    if constexpr (FEW) {
      met = met_of_few(choice, item / parts);
    } else {
      const int r = item / parts, begin = __builtin_amdgcn_readfirstlane(sorted.begin[r]);
      met.expert = __builtin_amdgcn_readfirstlane(sorted.experts[r]);
      met.n = __builtin_amdgcn_readfirstlane(sorted.begin[r + 1]) - begin;
      met.list = sorted.pairs + begin;
    }
    const int from = groups * part / parts * 4, to = groups * (part + 1) / parts * 4;
    float(*out)[16] = sums + part * pairs;
    for (int at = 0; at < met.n;) {
      if (MOST == 1 || met.n - at <= 16) {
        down_block<1, FEW>(m, met, at, c0, from, to, first, out);
        at += 16;
      } else {
        if constexpr (MOST == 2) down_block<2, FEW>(m, met, at, c0, from, to, first, out);
        at += 32;
      }
    }
  }
  float residual = 0.0f;
  const bool mine = tid < tokens * 16 && c0 + (tid & 15) < m.n_in;
  if (m.residual && mine) residual = value_at<DST>(m.residual, (int64_t)(t0 + (tid >> 4)) * m.residual_stride + c0 + (tid & 15));
  __syncthreads();
  for (int i = tid; i < tokens * 16; i += M_WAVES * WAVE) {
    const int t = i >> 4, c = c0 + (i & 15);
    if (c >= m.n_in) continue;
    float v = 0.0f;
    for (int j = 0; j < m.top_k; ++j) {
      const int pair = t * m.top_k + j;
      if (ids[pair] == NO_EXPERT) continue;
      float s = sums[pair][i & 15];
      for (int q = 1; q < parts; ++q) s += sums[q * pairs + pair][i & 15];
      v += weights[pair] * s;
    }
    if (m.residual) v += i == tid ? residual : value_at<DST>(m.residual, (int64_t)(t0 + t) * m.residual_stride + c);
    const int64_t at = (int64_t)(t0 + t) * m.y_stride + c;
    if (DST == QR_BF16) reinterpret_cast<uint16_t*>(m.y)[at] = bf16_bits(v);
    else reinterpret_cast<float*>(m.y)[at] = v;
  }
}

// ---------------------------------------------------------------------------
// launches

struct RoutePlan {
  bool rough, wide;
  int expert_tiles, token_tiles, splits;
};

// Rough logits where there is much to multiply; tiles of 32 x 32 where they fill
// the chip, or of 16 x 16; and the sum split until there are some 256 workgroups.
// Measured, us (8 of 256 experts, 7168 values): 512 tokens in 64 bits 49.5, rough
// 49.5; 1024 74 and 56, 2048 132 and 69, 4096 254 and 114; 8 of 512, 4096 values:
// 512 tokens 50 and 53, 1024 85 and 52.
RoutePlan route_plan(bool rough, int64_t n_experts, int64_t n_tok, int64_t n_in) {
  RoutePlan r;
  r.rough = rough && n_experts * n_tok > ((int64_t)1 << 30) / n_in;
  r.wide = !r.rough && ((n_experts + 31) / 32) * ((n_tok + 31) / 32) >= 256;
  const int64_t experts = r.rough ? ROUGH_E : r.wide ? 32 : 16, tokens = r.rough ? ROUGH_T : r.wide ? 32 : 16;
  r.expert_tiles = (int)((n_experts + experts - 1) / experts);
  r.token_tiles = (int)((n_tok + tokens - 1) / tokens);
  // (a part of the sum has eight waves' chunks, or four steps)
  const int64_t part = r.rough ? 4 * ROUGH_K : R_CHUNK * R_WAVES;
  const int64_t most = (n_in + part - 1) / part;
  int64_t s = 256 / ((int64_t)r.expert_tiles * r.token_tiles);
  s = s > R_SPLITS ? R_SPLITS : s;
  s = s > most ? most : s;
  r.splits = (int)(s < 1 ? 1 : s);
  return r;
}

size_t route_bytes(const RoutePlan& r, int64_t n_experts, int64_t n_tok) {
  const size_t logits = (size_t)r.splits * (size_t)n_tok * (size_t)n_experts * sizeof(double);
  return logits + (r.rough ? (size_t)r.splits * (size_t)(n_tok + n_experts) * sizeof(float) : 0);
}

template <int J>
int launch_choose(const Route& p, bool rough, hipStream_t s) {
  if constexpr (J > 1) {         // (rough logits are those of more than 64 experts)
    if (rough) {
      hipLaunchKernelGGL((k_route_settle<J>), dim3((uint32_t)p.n_tok), dim3(256), 0, s, p);
      return qr_check_launch("k_route_settle");
    }
  }
  hipLaunchKernelGGL((k_route_choose<J>), dim3((uint32_t)((p.n_tok + 3) / 4)), dim3(256), 0, s, p);
  return qr_check_launch("k_route_choose");
}

template <int SRC, int WSRC>
int launch_route(const Route& p, const RoutePlan& r, hipStream_t s) {
  // Few tokens of a router that one workgroup reads without being the last to end.
  // Measured, us (captured; a launch saved is worth some 3 more otherwise), first:
  // 8 experts of 4096 values, 1 token 4.9 / 6.7, 256 5.5 / 7.5, 1024 10.8 / 9.2;
  // 16 of 4096, 1 token 6.7 / 7.1, 256 7.6 / 8.1, 512 10.4 / 8.3; 32 of 2048, 1
  // token 7.0 / 6.4; 64 of 2048 10.8 / 7.0
  if (p.n_experts <= SMALL_EXPERTS && p.n_tok <= 256 && (int64_t)p.n_experts * p.n_in <= 65536) {
    hipLaunchKernelGGL((k_route_small<SRC, WSRC>), dim3((uint32_t)p.n_tok), dim3(SMALL_WAVES * WAVE), 0, s, p);
    return qr_check_launch("k_route_small");
  }
  const dim3 grid((uint32_t)(r.expert_tiles * (int64_t)r.token_tiles * r.splits)), block(R_WAVES * WAVE);
  const bool rough = SRC == QR_BF16 && WSRC == QR_BF16 && r.rough;
  if (rough) hipLaunchKernelGGL(k_route_rough, grid, dim3(512), 0, s, p, r.expert_tiles, r.token_tiles);
  else if (r.wide) hipLaunchKernelGGL((k_route_logits<SRC, WSRC, 2, 2>), grid, block, 0, s, p, r.expert_tiles, r.token_tiles);
  else hipLaunchKernelGGL((k_route_logits<SRC, WSRC, 1, 1>), grid, block, 0, s, p, r.expert_tiles, r.token_tiles);
  const int rc = qr_check_launch(rough ? "k_route_rough" : "k_route_logits");
  if (rc != QR_OK) return rc;
  if (p.n_experts <= 64) return launch_choose<1>(p, rough, s);
  if (p.n_experts <= 256) return launch_choose<4>(p, rough, s);
  return p.n_experts <= 512 ? launch_choose<8>(p, rough, s) : launch_choose<16>(p, rough, s);
}

bool route_shapes(int64_t n_experts, int64_t n_tok, int64_t n_in) {
  return n_experts >= 1 && n_experts <= QR_MOE_MAX_EXPERTS && n_tok >= 0 && n_tok < 1 << 22 && n_in >= 1 && n_in <= QR_I8_MAX_IN;
}

bool valid_moe(const qr_moe* m) {
  return m && m->n_experts >= 1 && m->n_experts <= QR_MOE_MAX_EXPERTS && qr_i8_row_bytes(m->n_in) &&
         qr_i8_row_bytes(m->n_mid) && m->expert_rows >= m->n_mid && m->expert_rows <= INT64_MAX / 4 / QR_MOE_MAX_EXPERTS / QR_I8_MAX_IN;
}

bool valid_pairs(int64_t n_tok, int64_t top_k) {
  return top_k >= 1 && top_k <= QR_MOE_MAX_TOP_K && n_tok >= 0 && n_tok <= QR_MOE_MAX_PAIRS / top_k;
}

int64_t scale_pitch(int64_t blocks) { return (blocks + 3) / 4 * 4; }

// Bytes of the hidden codes, whole cache lines.
int64_t code_bytes(int64_t pairs, int64_t blocks) { return (pairs * blocks * M_BLOCK + 255) / 256 * 256; }

template <int DST>
int launch_moe(const Moe& m, hipStream_t s) {
  const int64_t pairs = (int64_t)m.n_tok * m.top_k;
  const int64_t met = pairs < m.n_experts ? pairs : m.n_experts;
  const dim3 grid((uint32_t)(met * m.blocks)), block(M_WAVES * WAVE);
  const int64_t each = (pairs + m.n_experts - 1) / m.n_experts;   // pairs of an expert on average
  const bool few = pairs <= 64;
  if (few) hipLaunchKernelGGL((k_moe_hidden<true>), grid, block, 0, s, m);
  else hipLaunchKernelGGL((k_moe_hidden<false>), grid, block, (size_t)pairs * 2 * sizeof(uint16_t), s, m);
  const int rc = qr_check_launch("k_moe_hidden");
  if (rc != QR_OK) return rc;
  const int tokens_each = D_SLOTS / m.top_k;
  const dim3 tiles((uint32_t)((m.n_in + 15) / 16) * (uint32_t)((m.n_tok + tokens_each - 1) / tokens_each));
  // 32 pairs at a time where experts have that many and their sums are long:
  // half as many workgroups fit on a CU then. Measured, us a layer, 16 first:
  // 8 experts of 11008, 8 pairs each 217 / 220, 16 290 / 279, 20 339 / 300, 32
  // 437 / 420; 64 experts of 1408, 12 each 203 / 202, 24 309 / 322, 48 446 / 492
  const bool wide = each > 12 && m.n_mid >= 4096;
  if (few) {
    if (wide) hipLaunchKernelGGL((k_moe_down<DST, 2, true>), tiles, block, 0, s, m, tokens_each);
    else hipLaunchKernelGGL((k_moe_down<DST, 1, true>), tiles, block, 0, s, m, tokens_each);
  } else {
    if (wide) hipLaunchKernelGGL((k_moe_down<DST, 2, false>), tiles, block, 0, s, m, tokens_each);
    else hipLaunchKernelGGL((k_moe_down<DST, 1, false>), tiles, block, 0, s, m, tokens_each);
  }
  return qr_check_launch("k_moe_down");
}

}  // namespace

extern "C" {

size_t qr_moe_route_workspace_bytes(int64_t n_experts, int64_t n_tok, int64_t n_in) {
  if (!route_shapes(n_experts, n_tok, n_in) || n_tok == 0) return 0;
  // enough for either way to the logits: which one is taken goes by types and scores
  const size_t a = route_bytes(route_plan(false, n_experts, n_tok, n_in), n_experts, n_tok);
  const size_t b = route_bytes(route_plan(true, n_experts, n_tok, n_in), n_experts, n_tok);
  return a > b ? a : b;
}

int qr_moe_route(int src, const void* x, int64_t x_stride, int wtype, const void* w, const float* bias,
                 int64_t n_experts, int64_t n_tok, int64_t n_in, int64_t top_k, int score, int renorm, float factor,
                 int32_t* ids, float* weights, void* workspace, size_t workspace_bytes, void* stream) {
  qr_clear_error();
  if (src != QR_F32 && src != QR_BF16) return qr_fail(QR_EINVAL_TYPE, "source type %d is not QR_F32 or QR_BF16", src);
  if (wtype != QR_F32 && wtype != QR_BF16) return qr_fail(QR_EINVAL_TYPE, "weight type %d is not QR_F32 or QR_BF16", wtype);
  if (score != QR_SCORE_SOFTMAX && score != QR_SCORE_SIGMOID) return qr_fail(QR_EINVAL_TYPE, "score %d is not one of QR_SCORE_*", score);
  if (n_experts < 1 || n_experts > QR_MOE_MAX_EXPERTS)
    return qr_fail(QR_EINVAL_SHAPE, "n_experts=%lld must be in 1..%d", (long long)n_experts, QR_MOE_MAX_EXPERTS);
  if (n_in < 1 || n_in > QR_I8_MAX_IN) return qr_fail(QR_EINVAL_SHAPE, "n_in=%lld must be in 1..%d", (long long)n_in, QR_I8_MAX_IN);
  if (top_k < 1 || top_k > n_experts || top_k > QR_MOE_MAX_TOP_K)
    return qr_fail(QR_EINVAL_SHAPE, "top_k=%lld must be in 1..min(n_experts, %d)", (long long)top_k, QR_MOE_MAX_TOP_K);
  if (n_tok < 0 || x_stride < n_in) return qr_fail(QR_EINVAL_SHAPE, "negative n_tok, or x_stride below n_in");
  if (!(factor - factor == 0.0f)) return qr_fail(QR_EINVAL_SHAPE, "factor must be finite");
  if (n_tok == 0) return QR_OK;
  if (!route_shapes(n_experts, n_tok, n_in) || x_stride > INT64_MAX / 4 / n_tok)
    return qr_fail(QR_EOVERFLOW, "n_tok or x_stride too large");
  if (!x || !w || !ids || !weights) return qr_fail(QR_EINVAL_PTR, "x, w, ids and weights must be non-NULL");
  if (!qr_aligned(x, src == QR_BF16 ? 2 : 4) || !qr_aligned(w, wtype == QR_BF16 ? 2 : 4) || !qr_aligned(bias, 4) ||
      !qr_aligned(ids, 4) || !qr_aligned(weights, 4))
    return qr_fail(QR_EINVAL_PTR, "x, w, bias, ids and weights must be aligned to their elements");
  const size_t need = qr_moe_route_workspace_bytes(n_experts, n_tok, n_in);
  if (!workspace || !qr_aligned(workspace, 256)) return qr_fail(QR_EINVAL_PTR, "workspace must be non-NULL and 256-byte aligned");
  if (workspace_bytes < need) return qr_fail(QR_EINVAL_SHAPE, "workspace has %zu bytes, %zu are needed", workspace_bytes, need);
  // Both sides bf16, no softmax whose scores meet a bias or are the weights as they
  // are (those hang on all of the logits), and experts enough, since an exact logit
  // costs as much as seven on the matrix cores. 4096 tokens, us, in 64 bits and
  // rough: 1 of 128 experts 81 and 48, 8 of 128 85 and 75, 8 of 192 119 and 81; but
  // 32 of 256 166 and 187, 6 of 64 (2048 values) 29 and 44
  const bool rough = src == QR_BF16 && wtype == QR_BF16 && (score == QR_SCORE_SIGMOID || (renorm && !bias)) &&
                     n_experts > 64 + 7 * top_k;
  const RoutePlan r = route_plan(rough, n_experts, n_tok, n_in);
  double* logits = reinterpret_cast<double*>(workspace);
  float* squares = reinterpret_cast<float*>(logits + (size_t)r.splits * (size_t)n_tok * (size_t)n_experts);
  const Route p = {x, w, bias, logits, squares, ids, weights, x_stride, (int)n_experts, (int)n_tok,
                   (int)n_in, (int)top_k, r.splits, score, renorm, factor};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (src == QR_BF16) return wtype == QR_BF16 ? launch_route<QR_BF16, QR_BF16>(p, r, s) : launch_route<QR_BF16, QR_F32>(p, r, s);
  return wtype == QR_BF16 ? launch_route<QR_F32, QR_BF16>(p, r, s) : launch_route<QR_F32, QR_F32>(p, r, s);
}

size_t qr_moe_i8_workspace_bytes(const qr_moe* m, int64_t n_tok, int64_t top_k) {
  if (!valid_moe(m) || !valid_pairs(n_tok, top_k)) return 0;
  const int64_t pairs = n_tok * top_k, blocks = (m->n_mid + M_BLOCK - 1) / M_BLOCK;
  return (size_t)(code_bytes(pairs, blocks) + pairs * scale_pitch(blocks) * (int64_t)sizeof(float));
}

int qr_moe_i8(const qr_moe* m, const int8_t* x, const float* xd, const int32_t* ids, const float* weights,
              int64_t n_tok, int64_t top_k, int act, const void* residual, int64_t residual_stride, int dst, void* y,
              int64_t y_stride, void* workspace, size_t workspace_bytes, void* stream) {
  qr_clear_error();
  if (!valid_moe(m))
    return qr_fail(QR_EINVAL_SHAPE, "the experts must number 1..%d, n_in and n_mid lie in 1..%d, expert_rows not below n_mid",
                   QR_MOE_MAX_EXPERTS, QR_I8_MAX_IN);
  if (dst != QR_F32 && dst != QR_BF16) return qr_fail(QR_EINVAL_TYPE, "output type %d is not QR_F32 or QR_BF16", dst);
  if (act < QR_ACT_NONE || act > QR_ACT_GELU_TANH) return qr_fail(QR_EINVAL_TYPE, "activation %d is not one of QR_ACT_*", act);
  if (top_k < 1 || top_k > QR_MOE_MAX_TOP_K) return qr_fail(QR_EINVAL_SHAPE, "top_k=%lld must be in 1..%d", (long long)top_k, QR_MOE_MAX_TOP_K);
  if (n_tok < 0 || y_stride < m->n_in || (residual && residual_stride < m->n_in))
    return qr_fail(QR_EINVAL_SHAPE, "negative n_tok, or y_stride or residual_stride below n_in");
  if (n_tok == 0) return QR_OK;
  if (!valid_pairs(n_tok, top_k)) return qr_fail(QR_EOVERFLOW, "n_tok * top_k must be at most %d", QR_MOE_MAX_PAIRS);
  if (y_stride > INT64_MAX / 4 / n_tok || (residual && residual_stride > INT64_MAX / 4 / n_tok))
    return qr_fail(QR_EOVERFLOW, "y_stride or residual_stride too large");
  if (!m->gate || !m->up || !m->down || !m->gated || !m->upd || !m->downd || !x || !xd || !ids || !weights || !y)
    return qr_fail(QR_EINVAL_PTR, "the experts' arrays, x, xd, ids, weights and y must be non-NULL");
  const int64_t esize = dst == QR_BF16 ? 2 : 4;
  if (!qr_aligned(m->gate, 16) || !qr_aligned(m->up, 16) || !qr_aligned(m->down, 16) || !qr_aligned(m->gated, 4) ||
      !qr_aligned(m->upd, 4) || !qr_aligned(m->downd, 4) || !qr_aligned(x, 16) || !qr_aligned(xd, 4) || !qr_aligned(ids, 4) ||
      !qr_aligned(weights, 4) || !qr_aligned(y, (uintptr_t)esize) || !qr_aligned(residual, (uintptr_t)esize))
    return qr_fail(QR_EINVAL_PTR, "codes must be 16-byte aligned, everything else to its elements");
  const size_t need = qr_moe_i8_workspace_bytes(m, n_tok, top_k);
  if (!workspace || !qr_aligned(workspace, 256)) return qr_fail(QR_EINVAL_PTR, "workspace must be non-NULL and 256-byte aligned");
  if (workspace_bytes < need) return qr_fail(QR_EINVAL_SHAPE, "workspace has %zu bytes, %zu are needed", workspace_bytes, need);
  const int64_t row = m->n_in * esize, pairs = n_tok * top_k, in_bytes = (int64_t)qr_i8_row_bytes(m->n_in);
  if (residual && !(residual == y && (n_tok == 1 || residual_stride == y_stride)) &&
      rows_meet(y, y_stride * esize, residual, residual_stride * esize, row, n_tok))
    return qr_fail(QR_EINVAL_PTR, "y and residual must be the same rows or not overlap");
  if (rows_meet_range(y, y_stride * esize, row, n_tok, x, n_tok * in_bytes) ||
      rows_meet_range(y, y_stride * esize, row, n_tok, xd, n_tok * 4) ||
      rows_meet_range(y, y_stride * esize, row, n_tok, ids, pairs * 4) ||
      rows_meet_range(y, y_stride * esize, row, n_tok, weights, pairs * 4) ||
      rows_meet_range(y, y_stride * esize, row, n_tok, workspace, (int64_t)need))
    return qr_fail(QR_EINVAL_PTR, "y must not overlap x, xd, ids, weights or the workspace");
  if (rows_meet_range(workspace, (int64_t)need, (int64_t)need, 1, x, n_tok * in_bytes) ||
      rows_meet_range(workspace, (int64_t)need, (int64_t)need, 1, xd, n_tok * 4) ||
      rows_meet_range(workspace, (int64_t)need, (int64_t)need, 1, ids, pairs * 4) ||
      rows_meet_range(workspace, (int64_t)need, (int64_t)need, 1, weights, pairs * 4) ||
      (residual && rows_meet_range(residual, residual_stride * esize, row, n_tok, workspace, (int64_t)need)))
    return qr_fail(QR_EINVAL_PTR, "the workspace must not overlap x, xd, ids, weights or residual");
  const int64_t blocks = (m->n_mid + M_BLOCK - 1) / M_BLOCK;
  int8_t* h = reinterpret_cast<int8_t*>(workspace);
  const Moe a = {m->gate, m->up, m->down, m->gated, m->upd, m->downd, x, xd, ids, weights, h,
                 reinterpret_cast<float*>(h + code_bytes(pairs, blocks)), residual, y, m->expert_rows, residual_stride,
                 y_stride, (int)m->n_experts, (int)m->n_in, (int)m->n_mid, (int)in_bytes,
                 (int)qr_i8_row_bytes(m->n_mid), (int)blocks, (int)scale_pitch(blocks), (int)n_tok, (int)top_k, act};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dst == QR_BF16 ? launch_moe<QR_BF16>(a, s) : launch_moe<QR_F32>(a, s);
}

}  // extern "C"
