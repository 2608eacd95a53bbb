// serve_kv8.hip -- gfx950 kernels and C-ABI of the paged 8-bit key/value cache
// and of attention over it (declared in serve/qrow_kv8.h).

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "qr_internal.h"
#include "qrow.h"
#include "serve/qrow_kv8.h"
#include "serve_internal.h"

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 h16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 h16x8 __attribute__((ext_vector_type(8)));

constexpr int WAVE = 64;
constexpr int GROUP = 32;        // tokens of a V group: every block holds whole groups
constexpr int MAX_HEADS = 1024;

__device__ __forceinline__ float bf16_value(uint16_t h) { return __builtin_bit_cast(float, (uint32_t)h << 16); }

// fp32 to bf16, round to nearest even (NaN stays NaN).
__device__ __forceinline__ uint16_t bf16_bits(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

template <int SRC>
__device__ __forceinline__ float value_at(const void* x, int64_t i) {
  return SRC == QR_BF16 ? bf16_value(reinterpret_cast<const uint16_t*>(x)[i]) : reinterpret_cast<const float*>(x)[i];
}

template <int DST>
__device__ __forceinline__ void store_at(void* x, int64_t i, float v) {
  if (DST == QR_BF16) reinterpret_cast<uint16_t*>(x)[i] = bf16_bits(v);
  else reinterpret_cast<float*>(x)[i] = v;
}

// Four neighbouring outputs, at a multiple of four elements of an aligned array.
template <int DST>
__device__ __forceinline__ void store_heads(void* x, int64_t i, const f32x4& v) {
  if (DST == QR_BF16)
    *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(x) + i) =
        u32x2{(uint32_t)bf16_bits(v[0]) | (uint32_t)bf16_bits(v[1]) << 16,
              (uint32_t)bf16_bits(v[2]) | (uint32_t)bf16_bits(v[3]) << 16};
  else
    *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(x) + i) = v;
}

// The sequences of a call and the cache they live in.
struct Batch {
  const int32_t* cu;
  const int32_t* kv_len;
  const int32_t* table;
  int table_width, n_seq, n_tok;
};

struct Cache {
  int8_t* k;
  int8_t* v;
  float* kd;
  float* vd;
  int n_blocks, n_heads, shift;   // 2^shift tokens per block
};

// A sequence's rows and tokens. Rows [row0, row0 + n) of the call are the
// positions len - n ...
struct Span {
  int seq, row0, n, len;
};

__device__ __forceinline__ int clamp_row(const Batch& b, int r) { return r < 0 ? 0 : r > b.n_tok ? b.n_tok : r; }

// Which sequence a unit of work belongs to, without a table of units on the
// host: sequence s gets the units from floor(cu[s] * mul / 2^shift) + s * pad on,
// which leaves every sequence room for ceil(rows * mul / 2^shift) + pad - 1 units
// or more. A whole wave asks together: its lanes look at 64 sequences at once.
// Returns the unit's number within its sequence.
__device__ __forceinline__ int find_unit(const Batch& b, int64_t unit, int64_t mul, int shift, int pad, Span& sp) {
  const int lane = threadIdx.x & (WAVE - 1);
  int seq = -1, begin = 0, end = 0, len = 0;
  for (int base = 0; base < b.n_seq; base += WAVE) {
    // what the sequence's span needs is asked for with what finds it
    const int s = base + lane;
    int from = 0, to = 0, tokens = 0;
    if (s < b.n_seq) {
      from = clamp_row(b, b.cu[s]);
      to = clamp_row(b, b.cu[s + 1]);
      tokens = b.kv_len[s];
    }
    const uint64_t m = __ballot(s < b.n_seq && ((int64_t)from * mul >> shift) + (int64_t)s * pad <= unit);
    if (m != 0) {
      const int at = 63 - __builtin_clzll(m);
      seq = base + at;
      begin = __builtin_amdgcn_readlane(from, at);
      end = __builtin_amdgcn_readlane(to, at);
      len = __builtin_amdgcn_readlane(tokens, at);
    }
    if (m != ~0ull) break;
  }
  sp = {seq < 0 ? 0 : seq, begin, seq < 0 || end < begin ? 0 : end - begin, len};
  return (int)(unit - (((int64_t)begin * mul >> shift) + (int64_t)sp.seq * pad));
}

// The block in slot `slot` of a sequence's row of the table, or -1.
__device__ __forceinline__ int block_of(const int32_t* row, int width, int n_blocks, int slot) {
  if (slot < 0 || slot >= width) return -1;
  const int id = row[slot];
  return id >= 0 && id < n_blocks ? id : -1;
}

// Byte of channel d of token t in its V block.
template <int D>
__device__ __forceinline__ int v_byte(int t, int d) {
  return (t / GROUP) * (GROUP * D) + (d >> 1) * 64 + ((t % GROUP) >> 3) * 16 + (d & 1) * 8 + (t & 7);
}

// ---------------------------------------------------------------------------
// writing and reading

// The part of a sequence's rows that lies in one block: tokens [t0, t1) of
// the block are rows row .. row + (t1 - t0) - 1.
struct Piece {
  int id, t0, t1, row;
};

__device__ __forceinline__ Piece find_piece(const Batch& b, const Cache& c, int64_t unit) {
  Span sp;
  const int u = find_unit(b, unit, 1, c.shift, 2, sp);
  Piece p = {-1, 0, 0, 0};
  const int64_t first = (int64_t)sp.len - sp.n;         // position of the first row, may be negative
  const int64_t from = first < 0 ? 0 : first;
  const int64_t slot = (from >> c.shift) + u;
  const int64_t lo = slot << c.shift;
  if (u < 0 || sp.n == 0 || lo >= sp.len) return p;
  p.id = slot < b.table_width
             ? block_of(b.table + (int64_t)sp.seq * b.table_width, b.table_width, c.n_blocks, (int)slot)
             : -1;
  p.t0 = (int)(from > lo ? from - lo : 0);
  const int block = 1 << c.shift;
  p.t1 = (int)(sp.len - lo < block ? sp.len - lo : block);
  p.row = (int)(sp.row0 + (lo + p.t0 - first));
  return p;
}

// A workgroup takes the keys or the values of one head in one block. A thread
// takes squares of 8 tokens x 8 channels: rows of 16 or 32 bytes on the side
// of the caller's tensors, and on the side of the cache 8 codes of a token
// (keys) or 8 tokens of a channel (values), turned in registers. Up to four
// waves, and as many squares per thread as the block then needs; lanes are
// dealt so that neighbours meet neighbouring bytes on both sides.
constexpr int RW_THREADS = 256;

template <int D>
constexpr int squares_of(int block) { return block * D / 64; }

template <int D>
constexpr int rw_threads(int block) {
  return squares_of<D>(block) < WAVE ? WAVE : squares_of<D>(block) > RW_THREADS ? RW_THREADS : squares_of<D>(block);
}

// Square number `at`: its first token and channel in the block.
template <int D, bool VALUES>
__device__ __forceinline__ void square(int at, int& t, int& ch) {
  if (VALUES) {   // the four eights of a group first: 64 bytes of a pair of channels
    t = (at / (D / 2)) * GROUP + (at & 3) * 8;
    ch = at % (D / 2) / 4 * 8;
  } else {
    t = at / (D / 8) * 8;
    ch = at % (D / 8) * 8;
  }
}

template <int SRC>
__device__ __forceinline__ void load_heads8(const void* x, int64_t i, float (&v)[8]) {
  if (SRC == QR_BF16) {
    const u16x8 h = *reinterpret_cast<const u16x8*>(reinterpret_cast<const uint16_t*>(x) + i);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = bf16_value(h[k]);
  } else {
    const f32x4* p = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(x) + i);
    const f32x4 a = p[0], b = p[1];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = a[k];
      v[4 + k] = b[k];
    }
  }
}

__device__ __forceinline__ int code_of(float x) {
  return (int)__builtin_amdgcn_fmed3f(__builtin_rintf(x), -127.0f, 127.0f);
}

__device__ __forceinline__ int code_at(const u32x2& w, int i) { return (int8_t)(w[i >> 2] >> (8 * (i & 3))); }

__device__ __forceinline__ u32x2 pack8(const int (&q)[8]) {
  u32x2 w;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a = __builtin_amdgcn_perm((uint32_t)q[4 * h + 1], (uint32_t)q[4 * h], 0x0c0c0400u);
    const uint32_t b = __builtin_amdgcn_perm((uint32_t)q[4 * h + 3], (uint32_t)q[4 * h + 2], 0x0c0c0400u);
    w[h] = a | b << 16;
  }
  return w;
}

// How a block's scale changes with the new tokens, whose largest magnitude (as
// bits) one thread of the workgroup knows as `top`.
struct Growth {
  float inv, ratio;   // factors of new values and of old codes
  bool bad, grown;
};

__device__ __forceinline__ Growth grow(uint32_t top, int t0, float* scale, uint32_t* wave_max) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)top, s);
    top = o > top ? o : top;
  }
  if ((tid & (WAVE - 1)) == 0) wave_max[tid / WAVE] = top;
  const float old = t0 > 0 ? *scale : 0.0f;
  __syncthreads();   // every thread has read the old scale
  for (int w = 0; w < (int)blockDim.x / WAVE; ++w) top = wave_max[w] > top ? wave_max[w] : top;
  float cand = __builtin_bit_cast(float, top) / 127.0f;
  if (!(1.0f / cand < __builtin_inff())) cand = 0.0f;
  Growth g;
  g.bad = top >= 0x7f800000u || old != old;
  const float d = g.bad ? __builtin_nanf("") : old > cand ? old : cand;
  g.inv = 1.0f / d;
  if (g.bad || !(g.inv < __builtin_inff())) g.inv = 0.0f;
  g.grown = t0 > 0 && !g.bad && d > old;
  g.ratio = g.grown ? old / d : 1.0f;
  if (tid == 0) *scale = d;
  return g;
}

// A few tokens (a decode step): bound by the time from one load to the next
// and by fetching the code itself, so that loops stay loops; eight codes at a
// time, of one token for keys, of one channel for values. One token into each
// of 32 sequences, 8 heads of 128: 5 us (by squares 3 us more).
constexpr int FEW_TOKENS = 4;

template <int SRC, int D, bool VALUES>
__device__ __forceinline__ void append_few(const Cache& c, const Piece& p, int head, const void* __restrict__ x,
                                           int64_t stride, uint32_t* wave_max) {
  const int tid = threadIdx.x, threads = blockDim.x;
  const int64_t x0 = (int64_t)p.row * stride + (int64_t)head * D;
  uint32_t top = 0;
#pragma unroll 1
  for (int e = tid; e < (p.t1 - p.t0) * D; e += threads) {
    const uint32_t m =
        __builtin_bit_cast(uint32_t, value_at<SRC>(x, x0 + (int64_t)(e / D) * stride + e % D)) & 0x7fffffffu;
    top = m > top ? m : top;
  }
  const int64_t at_scale = (int64_t)p.id * c.n_heads + head;
  const Growth g = grow(top, p.t0, (VALUES ? c.vd : c.kd) + at_scale, wave_max);
  int8_t* codes = (VALUES ? c.v : c.k) + (at_scale << c.shift) * D;
  const int first = g.grown ? 0 : p.t0;   // tokens first .. t1 - 1 get codes
  const int n = VALUES ? ((p.t1 + 7) / 8 - first / 8) * D : (p.t1 - first) * (D / 8);
#pragma unroll 1
  for (int e = tid; e < n; e += threads) {
    const int t = VALUES ? (first / 8 + e / D) * 8 : first + e / (D / 8), ch = VALUES ? e % D : e % (D / 8) * 8;
    u32x2* to = reinterpret_cast<u32x2*>(codes + (VALUES ? v_byte<D>(t, ch) : t * D + ch));
    const u32x2 was = *to;
    int q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int ti = VALUES ? t + i : t, ci = VALUES ? ch : ch + i;
      q[i] = code_at(was, i);   // a token before an unchanged scale, or one behind the new ones
      if (ti < p.t0) {
        if (g.grown) q[i] = code_of((float)q[i] * g.ratio);
      } else if (ti < p.t1) {
        q[i] = g.bad ? 0 : code_of(value_at<SRC>(x, x0 + (int64_t)(ti - p.t0) * stride + ci) * g.inv);
      }
    }
    *to = pack8(q);
  }
}

// Each new value is read once and stays in registers between the block's
// maximum and its codes: bound by those bytes (12545 bf16 tokens of 8 heads of
// 128: 22.8 us, 3.4 TB/s; by single elements, read twice: 45 us).
template <int SRC, int D, int SQ, bool VALUES>
__device__ __forceinline__ void append_piece(const Cache& c, const Piece& p, int head, const void* __restrict__ x,
                                             int64_t stride, uint32_t* wave_max) {
  const int tid = threadIdx.x, n_squares = (D << c.shift) / 64;
  const int64_t x0 = (int64_t)p.row * stride + (int64_t)head * D;
  float v[SQ][8][8];
  uint32_t top = 0;
#pragma unroll
  for (int s = 0; s < SQ; ++s) {
    const int at = tid + s * (int)blockDim.x;
    int t, ch;
    square<D, VALUES>(at, t, ch);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (at < n_squares && t + k >= p.t0 && t + k < p.t1) {
        load_heads8<SRC>(x, x0 + (int64_t)(t + k - p.t0) * stride + ch, v[s][k]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[s][k][i] = 0.0f;
      }
    }
  }
#pragma unroll
  for (int s = 0; s < SQ; ++s)
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t m = __builtin_bit_cast(uint32_t, v[s][k][i]) & 0x7fffffffu;
        top = m > top ? m : top;
      }
  const int64_t at_scale = (int64_t)p.id * c.n_heads + head;
  int8_t* codes = (VALUES ? c.v : c.k) + (at_scale << c.shift) * D;
  // values: eight tokens share a word pair, so that squares at the ends keep
  // what the neighbouring tokens hold
  u32x4 was4[SQ][4];
  if (VALUES) {
#pragma unroll
    for (int s = 0; s < SQ; ++s) {
      const int at = tid + s * (int)blockDim.x;
      int t, ch;
      square<D, VALUES>(at, t, ch);
      const bool ends = at < n_squares && t < p.t1 && (t < p.t0 || t + 8 > p.t1);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        was4[s][i] = ends ? *reinterpret_cast<const u32x4*>(codes + v_byte<D>(t, ch + 2 * i)) : u32x4{};
    }
  }
  const Growth g = grow(top, p.t0, (VALUES ? c.vd : c.kd) + at_scale, wave_max);
  const int first = g.grown ? 0 : p.t0;   // tokens first .. t1 - 1 get codes
#pragma unroll
  for (int s = 0; s < SQ; ++s) {
    const int at = tid + s * (int)blockDim.x;
    int t, ch;
    square<D, VALUES>(at, t, ch);
    if (at >= n_squares || t + 8 <= first || t >= p.t1) continue;
    if (!VALUES) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (t + k < first || t + k >= p.t1) continue;
        u32x2* to = reinterpret_cast<u32x2*>(codes + (t + k) * D + ch);
        int q[8];
        if (t + k < p.t0) {
          const u32x2 was = *to;
#pragma unroll
          for (int i = 0; i < 8; ++i) q[i] = code_of((float)code_at(was, i) * g.ratio);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) q[i] = g.bad ? 0 : code_of(v[s][k][i] * g.inv);
        }
        *to = pack8(q);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        u32x4* to = reinterpret_cast<u32x4*>(codes + v_byte<D>(t, ch + i));
        const u32x4 was = was4[s][i / 2];
        u32x2 w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x2 old8 = {was[2 * h], was[2 * h + 1]};
          int q[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (t + k < p.t0) q[k] = g.grown ? code_of((float)code_at(old8, k) * g.ratio) : code_at(old8, k);
            else if (t + k >= p.t1) q[k] = code_at(old8, k);   // behind the new tokens
            else q[k] = g.bad ? 0 : code_of(v[s][k][i + h] * g.inv);
          }
          w[h] = pack8(q);
        }
        *to = u32x4{w[0][0], w[0][1], w[1][0], w[1][1]};
      }
    }
  }
}

template <int SRC, int D, int SQ>
__global__ __launch_bounds__(RW_THREADS) void k_kv8_append(Cache c, Batch b, const void* __restrict__ k,
                                                           const void* __restrict__ v, int64_t k_stride,
                                                           int64_t v_stride) {
  __shared__ uint32_t wave_max[RW_THREADS / WAVE];
  const Piece p = find_piece(b, c, blockIdx.x / c.n_heads);
  if (p.id < 0 || p.t1 <= p.t0) return;
  const int head = blockIdx.x % c.n_heads;
  if (p.t1 - p.t0 <= FEW_TOKENS) {
    if (blockIdx.y == 0) append_few<SRC, D, false>(c, p, head, k, k_stride, wave_max);
    else append_few<SRC, D, true>(c, p, head, v, v_stride, wave_max);
  } else if (blockIdx.y == 0) append_piece<SRC, D, SQ, false>(c, p, head, k, k_stride, wave_max);
  else {
    append_piece<SRC, D, SQ, true>(c, p, head, v, v_stride, wave_max);
  }
}

template <int DST>
__device__ __forceinline__ void store_heads8(void* x, int64_t i, const float (&v)[8]) {
  store_heads<DST>(x, i, f32x4{v[0], v[1], v[2], v[3]});
  store_heads<DST>(x, i + 4, f32x4{v[4], v[5], v[6], v[7]});
}

template <int DST, int D, bool VALUES>
__device__ __forceinline__ void read_piece(const Cache& c, const Piece& p, int head, void* __restrict__ x,
                                           int64_t stride) {
  const int tid = threadIdx.x, n_squares = (D << c.shift) / 64;
  const int64_t x0 = (int64_t)p.row * stride + (int64_t)head * D;
  const int64_t at_scale = (int64_t)(p.id < 0 ? 0 : p.id) * c.n_heads + head;
  const float d = p.id < 0 ? 0.0f : (VALUES ? c.vd : c.kd)[at_scale];
  const int8_t* codes = (VALUES ? c.v : c.k) + (at_scale << c.shift) * D;
  for (int at = tid; at < n_squares; at += (int)blockDim.x) {
    int t, ch;
    square<D, VALUES>(at, t, ch);
    if (t + 8 <= p.t0 || t >= p.t1) continue;
    u32x2 w[8] = {};   // of token k (keys), of channel ch + k (values)
    if (p.id >= 0) {
      if (VALUES) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const u32x4 two = *reinterpret_cast<const u32x4*>(codes + v_byte<D>(t, ch + i));
          w[i] = u32x2{two[0], two[1]};
          w[i + 1] = u32x2{two[2], two[3]};
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = *reinterpret_cast<const u32x2*>(codes + (t + k) * D + ch);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (t + k < p.t0 || t + k >= p.t1) continue;
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = p.id < 0 ? 0.0f : (float)(VALUES ? code_at(w[i], k) : code_at(w[k], i)) * d;
      store_heads8<DST>(x, x0 + (int64_t)(t + k - p.t0) * stride + ch, f);
    }
  }
}

// The decoder, over the same pieces: bound by the values it writes (12545
// tokens of 8 heads of 128 to fp32: 25.4 us, 5.1 TB/s).
template <int DST, int D>
__global__ __launch_bounds__(RW_THREADS) void k_kv8_read(Cache c, Batch b, void* __restrict__ k, void* __restrict__ v,
                                                         int64_t k_stride, int64_t v_stride) {
  const int tid = threadIdx.x, unit = blockIdx.x / c.n_heads, head = blockIdx.x % c.n_heads;
  const Piece p = find_piece(b, c, unit);
  if (p.t1 > p.t0) {
    if (blockIdx.y == 0) read_piece<DST, D, false>(c, p, head, k, k_stride);
    else read_piece<DST, D, true>(c, p, head, v, v_stride);
  }
  // rows before position 0: the sequence's first unit clears them
  Span sp;
  if (find_unit(b, unit, 1, c.shift, 2, sp) == 0 && sp.len < sp.n) {
    void* x = blockIdx.y == 0 ? k : v;
    const int64_t stride = blockIdx.y == 0 ? k_stride : v_stride;
    const int64_t lost = sp.len < 0 ? sp.n : (int64_t)sp.n - sp.len;
    for (int64_t e = tid; e < lost * D; e += blockDim.x)
      store_at<DST>(x, (sp.row0 + e / D) * stride + (int64_t)head * D + e % D, 0.0f);
  }
}

// ---------------------------------------------------------------------------
// attention

// Four codes to four fp16 values, exactly: the byte u = code + 128 in the low
// bits of 1024 (0x6400), minus 1152.
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const h16x2 bias = {(_Float16)1152.0f, (_Float16)1152.0f};
  const uint32_t a = __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u);
  const uint32_t b = __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u);
  lo = __builtin_bit_cast(uint32_t, __builtin_bit_cast(h16x2, a) - bias);
  hi = __builtin_bit_cast(uint32_t, __builtin_bit_cast(h16x2, b) - bias);
}

__device__ __forceinline__ h16x8 codes8(uint32_t w0, uint32_t w1) {
  u32x4 r;
  uint32_t a, b;
  codes_to_half(w0, a, b);
  r[0] = a;
  r[1] = b;
  codes_to_half(w1, a, b);
  r[2] = a;
  r[3] = b;
  return __builtin_bit_cast(h16x8, r);
}

struct Attention {
  const void* q;
  void* out;
  float* part;       // [units][heads][splits] x (rows of D values, their maxima, their sums)
  int64_t q_stride, out_stride;
  float scale;       // times log2(e)
  int64_t window;
  int group;         // query heads per key/value head
  int n_splits, n_units;
};

constexpr int A_SHIFT = 4, A_ROWS = 1 << A_SHIFT;   // rows of a unit
constexpr int A_WAVES = 4;
constexpr int A_MIN_GROUPS = 8;  // token groups a split is worth (both kernels)
constexpr float NEG_INF = -__builtin_inff();
// Weights are exp2(s - max + 10): the largest is 2^10, so that small ones keep
// more of their bits in fp16, whose normal range ends at 2^-14.
constexpr float P_SHIFT = 10.0f;

// The visible tiles (of 32 `ng` tokens) of a unit and their share for one split.
struct Range {
  int g0, n, per, used;   // first group of the first tile, tiles, tiles per split, splits that have any
};

__device__ __forceinline__ Range visible(const Span& sp, int first_row, int rows, const Attention& a, int64_t limit,
                                         int ng) {
  Range r = {0, 0, 0, 0};
  if (rows <= 0) return r;
  int64_t last = (int64_t)sp.len - sp.n + (first_row + rows - 1) / a.group;
  if (last >= limit) last = limit - 1;
  int64_t from = 0;
  if (a.window > 0) {
    from = (int64_t)sp.len - sp.n + first_row / a.group - a.window + 1;
    if (from < 0) from = 0;
  }
  if (last < from) return r;
  const int tile = (int)(from / (GROUP * ng));
  r.g0 = tile * ng;
  r.n = (int)(last / (GROUP * ng)) - tile + 1;
  r.per = (r.n + a.n_splits - 1) / a.n_splits;
  if (r.per < A_MIN_GROUPS / ng) r.per = A_MIN_GROUPS / ng;
  r.used = (r.n + r.per - 1) / r.per;
  return r;
}

// A float of one lane, for all.
__device__ __forceinline__ float lane_value(float x, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}

// Eight query values of one row as fp16 operands: the row is scaled by 2^-e
// (its largest magnitude then lies in [2^13, 2^14)), and fp32 rows keep a
// second part for the bits that the first one lost.
template <int SRC>
__device__ __forceinline__ void query_half(const float (&x)[8], int e, h16x8& hi, h16x8& lo) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float f = __builtin_ldexpf(x[i], 14 - e);
    hi[i] = (_Float16)f;
    if (SRC == QR_F32) lo[i] = (_Float16)(f - (float)hi[i]);
  }
}

// Attention of 16 rows (a row is a token and one of the query heads of the
// key/value head) over one split of their tokens: single tokens, and chunks of
// a few. Four waves take the 32-token groups in turn; everything a wave needs
// of a group goes from memory straight into matrix operands, once, and the next group's codes
// are on their way while this one's are multiplied. Transposed products: S' =
// K Q', so that a lane holds eight neighbouring tokens of one row, which is
// what the second product, O' = V' P', takes as its right operand.
//
// Bound by the codes: one token each of 64 sequences of up to 8192, 32 heads
// over 8 of 128: 148 to 151 us by card, 4.8 TB/s (148 against 156 us with half
// the splits; without loading ahead a third more). 700 tokens of 4 sequences:
// 10.6 us, dependent loads.
template <int SRC, int D>
__global__ __launch_bounds__(A_WAVES * WAVE) void k_attention_kv8(Cache c, Batch b, Attention a) {
  constexpr int KS = D / 64;   // 64-channel steps of the first product
  constexpr int VS = D / 32;   // 32-channel steps of the second
  constexpr bool F32 = SRC == QR_F32;
  __shared__ float join_o[A_WAVES][A_ROWS][D + 4];
  __shared__ float join_m[A_WAVES][A_ROWS], join_l[A_WAVES][A_ROWS];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lg = lane >> 4;
  const int unit = blockIdx.x / c.n_heads, head = blockIdx.x % c.n_heads, split = blockIdx.y;

  Span sp;
  const int u = find_unit(b, unit, a.group, A_SHIFT, 1, sp);
  const int64_t n_rows = (int64_t)sp.n * a.group;
  const int64_t first_row = (int64_t)u * A_ROWS;
  if (u < 0 || first_row >= n_rows) return;
  const int rows = (int)(n_rows - first_row < A_ROWS ? n_rows - first_row : A_ROWS);
  const int64_t limit = (int64_t)b.table_width << c.shift;
  const Range vis = visible(sp, (int)first_row, rows, a, limit, 1);
  if (split > 0 && split >= vis.used) return;

  // this lane's row
  const int r = (int)first_row + (li < rows ? li : rows - 1);
  const int tok = sp.row0 + r / a.group;
  const int qh = head * a.group + r % a.group;
  const int64_t pos = (int64_t)sp.len - sp.n + r / a.group;
  const int64_t low = a.window > 0 ? pos - a.window : -1;   // positions above low, up to pos

  // queries
  h16x8 qhi[2 * KS], qlo[2 * KS];
  float row_scale;
  {
    float x[2 * KS][8];
    uint32_t top = 0;
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        load_heads8<SRC>(a.q, tok * a.q_stride + (int64_t)qh * D + 64 * s + 16 * lg + 8 * h, x[2 * s + h]);
#pragma unroll
    for (int s = 0; s < 2 * KS; ++s)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t m = __builtin_bit_cast(uint32_t, x[s][i]) & 0x7fffffffu;
        top = m > top ? m : top;
      }
#pragma unroll
    for (int s = 16; s < 64; s <<= 1) {
      const uint32_t o = (uint32_t)__shfl_xor((int)top, s);
      top = o > top ? o : top;
    }
    const bool bad = top >= 0x7f800000u;
    const float amax = bad ? 0.0f : __builtin_bit_cast(float, top);
    int e = 0;
    if (amax > 0.0f) (void)__builtin_frexpf(amax, &e);
#pragma unroll
    for (int s = 0; s < 2 * KS; ++s) query_half<SRC>(x[s], e, qhi[s], qlo[s]);
    row_scale = bad ? __builtin_nanf("") : __builtin_ldexpf(a.scale, e - 14);
  }

  f32x4 acc[2 * VS] = {};
  float m_run = NEG_INF, l_run = 0.0f;
  const int end = vis.g0 + (vis.n < (split + 1) * vis.per ? vis.n : (split + 1) * vis.per);
  const int begin = vis.g0 + split * vis.per + wave;
  // every row sees all tokens from clear_from up to clear_to
  const int64_t clear_to = (int64_t)sp.len - sp.n + first_row / a.group;
  const int64_t clear_from = a.window > 0 ? (int64_t)sp.len - sp.n + (first_row + rows - 1) / a.group - a.window + 1 : 0;

  // Blocks and scales of the wave's next 64 groups, one per lane; the codes of
  // the next group are loaded while this one's are multiplied.
  const int32_t* table_row = b.table + (int64_t)sp.seq * b.table_width;
  int ids = -1;
  float kds = 0.0f, vds = 0.0f;
  auto look_ahead = [&](int g) {
    const int mine = g + lane * A_WAVES;
    ids = mine < end ? block_of(table_row, b.table_width, c.n_blocks, mine >> (c.shift - 5)) : -1;
    if (ids >= 0) {
      kds = c.kd[(int64_t)ids * c.n_heads + head];
      vds = c.vd[(int64_t)ids * c.n_heads + head];
    }
  };
  u32x4 kw[2][KS], vw[VS];
  int id = -1;
  float kd = 0.0f, vd = 0.0f;
  auto fetch = [&](int it) {
    id = __builtin_amdgcn_readlane(ids, it);
    kd = lane_value(kds, it);
    vd = lane_value(vds, it);
  };
  auto load = [&](int g) {
    if (id < 0) return;
    const int64_t at = (((int64_t)id * c.n_heads + head) << c.shift) + (g * GROUP & ((1 << c.shift) - 1));
    const int8_t* kp = c.k + at * D;
    const int8_t* vp = c.v + at * D;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
        kw[t][ks] =
            *reinterpret_cast<const u32x4*>(kp + (8 * (li >> 2) + 4 * t + (li & 3)) * D + 16 * lg + 64 * ks);
#pragma unroll
    for (int vsx = 0; vsx < VS; ++vsx) vw[vsx] = *reinterpret_cast<const u32x4*>(vp + (16 * vsx + li) * 64 + 16 * lg);
  };
  look_ahead(begin);
  fetch(0);
  load(begin);
  for (int g = begin, it = 0; g < end; g += A_WAVES) {
    u32x4 kc[2][KS], vc[VS];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) kc[t][ks] = kw[t][ks];
#pragma unroll
    for (int vsx = 0; vsx < VS; ++vsx) vc[vsx] = vw[vsx];
    const bool have = id >= 0;
    const float kd_now = kd, vd_now = vd;
    if (++it == WAVE) {
      it = 0;
      look_ahead(g + A_WAVES);
    }
    fetch(it);
    load(g + A_WAVES);
    if (!have) continue;

    f32x4 s[2] = {};
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const h16x8 k0 = codes8(kc[t][ks][0], kc[t][ks][1]), k1 = codes8(kc[t][ks][2], kc[t][ks][3]);
        s[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, qhi[2 * ks], s[t], 0, 0, 0);
        s[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, qhi[2 * ks + 1], s[t], 0, 0, 0);
        if (F32) {
          s[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, qlo[2 * ks], s[t], 0, 0, 0);
          s[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, qlo[2 * ks + 1], s[t], 0, 0, 0);
        }
      }
    // scores of tokens t0 + 8 lg + i, in units of log 2
    const int64_t t0 = (int64_t)g * GROUP;
    const float f = row_scale * kd_now;
    float p[8];
    float top = NEG_INF;
    float vs = vd_now;
    if (t0 >= clear_from && t0 + GROUP - 1 <= clear_to) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = s[i >> 2][i & 3] * f;
        top = __builtin_fmaxf(top, p[i]);
      }
    } else {
      bool any = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t j = t0 + 8 * lg + i;
        const bool seen = j <= pos && j > low;
        p[i] = seen ? s[i >> 2][i & 3] * f : NEG_INF;
        top = __builtin_fmaxf(top, p[i]);
        any |= seen;
      }
      // a row that sees none of the group must not meet its value scale,
      // which may be NaN
      uint64_t sees = __ballot(any);
      sees |= sees >> 32;
      sees |= sees >> 16;
      if (!((sees >> li) & 1)) vs = 0.0f;
    }
    top = __builtin_fmaxf(top, __shfl_xor(top, 16));
    top = __builtin_fmaxf(top, __shfl_xor(top, 32));
    const float m_new = __builtin_fmaxf(m_run, top);
    const float ref = m_new == NEG_INF ? 0.0f : m_new - P_SHIFT;
    const float alpha = __builtin_amdgcn_exp2f(m_run - (m_new == NEG_INF ? 0.0f : m_new));
    m_run = m_new;
    float sum = 0.0f;
    h16x8 phi, plo;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = __builtin_amdgcn_exp2f(p[i] - ref);
      sum += p[i];
      phi[i] = (_Float16)p[i];
      if (F32) plo[i] = (_Float16)(p[i] - (float)phi[i]);
    }
    l_run = __builtin_fmaf(l_run, alpha, sum);
#pragma unroll
    for (int vsx = 0; vsx < VS; ++vsx) {
      const h16x8 v0 = codes8(vc[vsx][0], vc[vsx][1]), v1 = codes8(vc[vsx][2], vc[vsx][3]);
      f32x4 o0 = {}, o1 = {};
      o0 = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, phi, o0, 0, 0, 0);
      o1 = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, phi, o1, 0, 0, 0);
      if (F32) {
        o0 = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, plo, o0, 0, 0, 0);
        o1 = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, plo, o1, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * vsx][i] = __builtin_fmaf(o0[i], vs, acc[2 * vsx][i] * alpha);
        acc[2 * vsx + 1][i] = __builtin_fmaf(o1[i], vs, acc[2 * vsx + 1][i] * alpha);
      }
    }
  }
  l_run += __shfl_xor(l_run, 16);
  l_run += __shfl_xor(l_run, 32);

  // the waves' parts joined: lane (li, lg) holds channels 32 vs + 8 lg + 2 i +
  // (0, 1) of row li
#pragma unroll
  for (int vsx = 0; vsx < VS; ++vsx)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      join_o[wave][li][32 * vsx + 8 * lg + 2 * i] = acc[2 * vsx][i];
      join_o[wave][li][32 * vsx + 8 * lg + 2 * i + 1] = acc[2 * vsx + 1][i];
    }
  if (lg == 0) {
    join_m[wave][li] = m_run;
    join_l[wave][li] = l_run;
  }
  __syncthreads();
  for (int e = tid; e < rows * D; e += A_WAVES * WAVE) {
    const int row = e / D, ch = e % D;
    float m = NEG_INF;
#pragma unroll
    for (int w = 0; w < A_WAVES; ++w) m = __builtin_fmaxf(m, join_m[w][row]);
    const float ref = m == NEG_INF ? 0.0f : m;
    float o = 0.0f, l = 0.0f;
#pragma unroll
    for (int w = 0; w < A_WAVES; ++w) {
      const float f = __builtin_amdgcn_exp2f(join_m[w][row] - ref);
      o = __builtin_fmaf(join_o[w][row][ch], f, o);
      l = __builtin_fmaf(join_l[w][row], f, l);
    }
    if (vis.used <= 1) {
      const int rr = (int)first_row + row;
      const int64_t at = (int64_t)(sp.row0 + rr / a.group) * a.out_stride + (int64_t)(head * a.group + rr % a.group) * D + ch;
      store_at<SRC>(a.out, at, l == 0.0f ? 0.0f : o / l);
    } else {
      float* part = a.part + (((int64_t)unit * c.n_heads + head) * a.n_splits + split) * A_ROWS * (D + 2);
      part[row * D + ch] = o;
      if (ch == 0) {
        part[A_ROWS * D + row] = m;
        part[A_ROWS * D + A_ROWS + row] = l;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// attention of many rows

constexpr int P_SHIFT_ROWS = 7, P_ROWS = 1 << P_SHIFT_ROWS;   // rows of a unit: 32 per wave
constexpr int P_WAVES = 4;
constexpr float P_LAZY = 5.0f;   // how far scores may pass the reference maximum

// The value scale of a group as (mantissa, exponent) for weights that carry
// it: 2^e * 2^lm = scale, inv = 2^-lm. A scale of zero gets an exponent far
// below all others, one that is not finite a NaN.
struct ValueScale {
  int e;
  float lm, inv;
};

constexpr int E_NONE = -100000;
// A weight carries the exponent of its value scale, from 2^0 to 2^-P_FOLD of
// the reference: with P_SHIFT, whose largest weight is 2^10, fp16 then still
// counts weights of 2^-31 of the largest (half its smallest step is 2^-25, and
// the scale's mantissa takes another 2^-1).
constexpr int P_FOLD = 3;
// How far the reference may lie below the largest scale met: outputs, below
// 2^53 of the reference (2^31 tokens of 127 * 2^15), then stay below 2^126.
constexpr int P_REACH = 73;

template <int V>
struct Index {
  static constexpr int value = V;
};

// Where a 16-byte piece lies in LDS: piece p of K row r at p ^ k_swizzle(r),
// channel d of the V tokens 8 e .. at d ^ v_swizzle(e). Sixteen lanes that read
// or write side by side then meet sixteen different pieces of 256 bytes. (The
// counters still show 83k conflict cycles per CU in the prompts' case below, a
// tenth of its time; which access they belong to is not known.)
template <int D>
__device__ __forceinline__ int k_swizzle(int r) { return D == 64 ? (r >> 1) & 7 : r & 15; }
__device__ __forceinline__ int v_swizzle(int e) { return (e & 1) << 3 | e >> 1; }

// The value that the lane 32 further (or nearer) holds.
__device__ __forceinline__ float other_half(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_bit_cast(float, (threadIdx.x & 32) ? r[0] : r[1]);
}

__device__ __forceinline__ ValueScale value_scale(float vd) {
  ValueScale v;
  const float m = __builtin_amdgcn_frexp_mantf(vd);   // [0.5, 1)
  v.e = vd > 0.0f ? __builtin_amdgcn_frexp_expf(vd) : E_NONE;
  v.lm = vd > 0.0f ? __builtin_amdgcn_logf(m) : 0.0f;
  v.inv = vd > 0.0f ? __builtin_amdgcn_rcpf(m) : 1.0f;
  if (!(vd < __builtin_inff())) {
    v.e = E_NONE;
    v.lm = __builtin_nanf("");
  }
  return v;
}

// Attention of 128 rows (32 per wave) over one split of their tokens, in
// tiles of 32 NG tokens. A tile's codes are turned into fp16 once, on their
// way into LDS, and every wave multiplies from there: S' = K Q', O' = V' P'.
// The rows of the K tile are placed so that the tokens which a lane gets from
// the first product are the ones that it brings to the second.
//
// The value scale of a group of 32 tokens goes into the exponent of its
// weights, relative to a power of two per wave (e_ref): no second pass over the
// outputs. Their sum takes the factor out again. The outputs are rescaled only
// when a score passes the reference maximum by 2^5 (the weights, at most 2^15,
// still fit fp16), or where a group's scale lies above e_ref or more than
// 2^P_FOLD below it: e_ref then follows, so that a group's weights keep their
// bits whatever the scales of others.
//
// Prompts of 4 sequences of up to 4096 tokens, 32 heads over 8 of 128: 455 to
// 488 us by card, 700 to 750 TFLOP/s. Of a SIMD's 915k busy cycles 333k are
// products, and its 119k vector instructions take four cycles each: together
// 809k, so that the two units seem to work in turn more than at once, with two
// waves a SIMD. Heads of a unit side by side: 12% off the time; blocks and
// scales looked up in lanes, not by every wave in every tile: 25%. Following
// the value scales down as well as up costs 2% (fp32: 5%). 64-token tiles (32
// for 256 channels, whose two buffers fill the same LDS) and 128 rows: 32-token
// tiles at three waves a SIMD took 20% longer, 256 rows in eight waves 2%.
template <int SRC, int D, int NG>
__global__ __launch_bounds__(P_WAVES * WAVE, D == 256 || (SRC == QR_F32 && D == 128) ? 1 : 2) void k_attention_kv8_rows(Cache c, Batch b, Attention a) {
  constexpr int THREADS = P_WAVES * WAVE;
  constexpr int KS = D / 16;                     // steps of the first product
  constexpr int DT = D / 32;                     // 32-channel tiles of the output
  constexpr int TOK = GROUP * NG;
  constexpr int CH = TOK * D / 16 / THREADS;     // 16-byte pieces per thread
  constexpr bool F32 = SRC == QR_F32;
  static_assert(CH >= 1 && TOK * D / 16 % THREADS == 0, "whole pieces");
  __shared__ __attribute__((aligned(16))) uint8_t lds_k[2][TOK * D * 2];
  __shared__ __attribute__((aligned(16))) uint8_t lds_v[2][TOK * D * 2];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 31, lh = lane >> 5;
  // the longest prefixes first, the heads of a unit side by side: with 8 heads
  // each XCD reads the keys and values of one
  const int unit = a.n_units - 1 - blockIdx.x / c.n_heads, head = blockIdx.x % c.n_heads, split = blockIdx.y;

  Span sp;
  const int u = find_unit(b, unit, a.group, P_SHIFT_ROWS, 1, sp);
  const int64_t n_rows = (int64_t)sp.n * a.group;
  const int64_t first_row = (int64_t)u * P_ROWS;
  if (u < 0 || first_row >= n_rows) return;
  const int rows = (int)(n_rows - first_row < P_ROWS ? n_rows - first_row : P_ROWS);
  const Range vis = visible(sp, (int)first_row, rows, a, (int64_t)b.table_width << c.shift, NG);
  if (split > 0 && split >= vis.used) return;

  // this lane's row; a wave behind the last row repeats it
  const int wrow = 32 * wave < rows ? 32 * wave : rows - 1;            // first row of the wave
  const int wlast = 32 * wave + 31 < rows ? 32 * wave + 31 : rows - 1;
  const int row = 32 * wave + li < rows ? 32 * wave + li : rows - 1;
  const int r = (int)first_row + row;
  const int tok = sp.row0 + r / a.group;
  const int qh = head * a.group + r % a.group;
  // positions fit 32 bits: they are below kv_len
  const int base = (int)((int64_t)sp.len - sp.n < INT32_MIN ? INT32_MIN : (int64_t)sp.len - sp.n);
  const int pos = base + r / a.group;
  auto window_of = [&](int p) { return a.window > 0 && (int64_t)p - a.window >= 0 ? (int)(p - a.window) : -1; };
  const int low = window_of(pos);   // the row sees low + 1 .. pos
  // all rows of the wave see the tokens clear_from .. clear_to, none sees any
  // outside any_from .. any_to
  const int clear_to = base + ((int)first_row + wrow) / a.group, any_to = base + ((int)first_row + wlast) / a.group;
  const int clear_from = window_of(any_to) + 1, any_from = window_of(clear_to) + 1;

  f32x16 acc[DT] = {};
  float m_run = NEG_INF, l_run = 0.0f;
  int e_ref = E_NONE, e_most = E_NONE;

  const int tile0 = vis.g0 / NG + split * vis.per;
  const int tile_end = vis.g0 / NG + (vis.n < (split + 1) * vis.per ? vis.n : (split + 1) * vis.per);

  // Blocks and scales of 64 groups from first_known on, one group per lane:
  // looked up once for many tiles, and read from the lane that holds them.
  const int32_t* table_row = b.table + (int64_t)sp.seq * b.table_width;
  int first_known, ids;
  float kds;
  ValueScale vds;
  auto look_up = [&](int tile) {
    first_known = tile * NG;
    const int g = first_known + lane;
    ids = g < tile_end * NG ? block_of(table_row, b.table_width, c.n_blocks, g >> (c.shift - 5)) : -1;
    float vd = 0.0f;
    kds = 0.0f;
    if (ids >= 0) {
      const int64_t at = (int64_t)ids * c.n_heads + head;
      kds = c.kd[at];
      vd = c.vd[at];
    }
    vds = value_scale(vd);
  };
  u32x4 rawk[CH] = {}, rawv[CH] = {};
  auto fetch = [&](int tile) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int at = tid + i * THREADS;
      const int g = tile * NG + __builtin_amdgcn_readfirstlane(at / (2 * D));   // group: 2 D pieces each
      const int id = __builtin_amdgcn_readlane(ids, g - first_known);
      if (id >= 0) {
        const int64_t from = ((((int64_t)id * c.n_heads + head) << c.shift) + (g * GROUP & ((1 << c.shift) - 1))) * D;
        rawk[i] = *reinterpret_cast<const u32x4*>(c.k + from + (at % (2 * D)) * 16);
        rawv[i] = *reinterpret_cast<const u32x4*>(c.v + from + (at % (2 * D)) * 16);
      }
    }
  };
  auto stage = [&](int buf) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int at = tid + i * THREADS;
      // keys: token t of the tile goes to row t with bits 2 and 3 exchanged
      const int t = at / (D / 16), piece = at % (D / 16) * 2;
      const int to = (t & ~12) | ((t & 4) << 1) | ((t & 8) >> 1);
      uint8_t* kr = lds_k[buf] + to * (2 * D);
      *reinterpret_cast<h16x8*>(kr + (piece ^ k_swizzle<D>(to)) * 16) = codes8(rawk[i][0], rawk[i][1]);
      *reinterpret_cast<h16x8*>(kr + ((piece + 1) ^ k_swizzle<D>(to)) * 16) = codes8(rawk[i][2], rawk[i][3]);
      // values: eight tokens of a channel, by group, eight, channel
      const int g = at / (2 * D), pair = at % (2 * D) / 4, eight = at % 4;
      uint8_t* vr = lds_v[buf] + (g * 4 + eight) * (D * 16);
      *reinterpret_cast<h16x8*>(vr + ((2 * pair) ^ v_swizzle(eight)) * 16) = codes8(rawv[i][0], rawv[i][1]);
      *reinterpret_cast<h16x8*>(vr + ((2 * pair + 1) ^ v_swizzle(eight)) * 16) = codes8(rawv[i][2], rawv[i][3]);
    }
  };

  // the first tile is on its way while the queries come in
  look_up(tile0);
  fetch(tile0);
  h16x8 qhi[KS], qlo[F32 ? KS : 1];
  float row_scale;
  {
    uint32_t top = 0;
    float x[KS][8];
#pragma unroll
    for (int s = 0; s < KS; ++s)
      load_heads8<SRC>(a.q, tok * a.q_stride + (int64_t)qh * D + 16 * s + 8 * lh, x[s]);
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t m = __builtin_bit_cast(uint32_t, x[s][i]) & 0x7fffffffu;
        top = m > top ? m : top;
      }
    const uint32_t o = (uint32_t)__shfl_xor((int)top, 32);
    top = o > top ? o : top;
    const bool bad = top >= 0x7f800000u;
    const float amax = bad ? 0.0f : __builtin_bit_cast(float, top);
    int e = 0;
    if (amax > 0.0f) (void)__builtin_frexpf(amax, &e);
    // the factor's sign goes to the queries: a maximum of scores is then the
    // maximum of products
    const float sign = a.scale < 0.0f ? -1.0f : 1.0f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[s][i] *= sign;
      h16x8 lo;
      query_half<SRC>(x[s], e, qhi[s], lo);
      if (F32) qlo[s] = lo;
    }
    row_scale = bad ? __builtin_nanf("") : __builtin_ldexpf(a.scale * sign, e - 14);
  }

  stage(0);
  fetch(tile0 + 1);
  __syncthreads();
  // One tile: the next one is staged into the other buffer, the one after
  // that is asked for, and this one multiplied.
  auto step = [&](int tile, auto buf_tag) {
    constexpr int BUF = decltype(buf_tag)::value;
    if ((tile + 3) * NG > first_known + WAVE) look_up(tile);
    const int tile_t0 = tile * TOK;
    const bool idle = tile_t0 > any_to || tile_t0 + TOK - 1 < any_from;
    f32x16 s[NG];
    if (!idle) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[g][i] = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const h16x8 ka = *reinterpret_cast<const h16x8*>(lds_k[BUF] + (g * GROUP + li) * (2 * D) +
                                                           ((2 * k + lh) ^ k_swizzle<D>(li)) * 16);
          s[g] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ka, qhi[k], s[g], 0, 0, 0);
          if (F32) s[g] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ka, qlo[k], s[g], 0, 0, 0);
        }
      }
    }
    // converting the next tile keeps the vector unit busy meanwhile
    if (tile + 1 < tile_end) {
      stage(BUF ^ 1);
      fetch(tile + 2);
    }
    if (idle) return;
    // s[g][i]: token t0 + 16 (i / 8) + 8 lh + i % 8 of this lane's row
    float f[NG], top = NEG_INF;
    float lm[NG], inv[NG];   // of the value scales, with their exponents
    int ex[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int t0 = tile_t0 + g * GROUP;
      // (a factor of zero becomes one that moves no score: -inf times it
      // stays -inf)
      const int from = tile * NG + g - first_known;
      const bool have = __builtin_amdgcn_readlane(ids, from) >= 0;
      f[g] = row_scale * lane_value(kds, from);
      f[g] = f[g] < 1e-30f ? 1e-30f : f[g];
      ex[g] = __builtin_amdgcn_readlane(vds.e, from);
      lm[g] = lane_value(vds.lm, from);
      inv[g] = lane_value(vds.inv, from);
      if (!have || t0 < clear_from || t0 + GROUP - 1 > clear_to) {
        // the row sees the group's tokens lo + 1 .. hi
        const int hi = have && pos >= t0 ? pos - t0 : -1, lo = low >= t0 ? low - t0 : -1;
        const int first = lo + 1 - 8 * lh;
        const uint32_t count = hi > lo ? hi - lo : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = 16 * (i >> 3) + (i & 7);
          s[g][i] = (uint32_t)(j - first) < count ? s[g][i] : NEG_INF;
        }
        const bool seen_any = hi >= 0 && lo < GROUP - 1;
        if (!seen_any) {   // the group's scales, which may be NaN, stay out
          f[g] = 1.0f;
          lm[g] = 0.0f;
        }
      }
      float t = s[g][0];
#pragma unroll
      for (int i = 1; i < 16; ++i) t = __builtin_elementwise_maximum(t, s[g][i]);
      t *= f[g];
      top = t > top ? t : top;
    }
    const float across = other_half(top);
    top = across > top ? across : top;
    // outputs to the new maximum, and to a reference that serves exponent e
    auto serves = [&](int e) { return (e <= e_ref) & ((e >= e_ref - P_FOLD) | (e == E_NONE)); };
    auto rescale = [&](int e) __attribute__((always_inline)) {
      const float m_new = top > m_run ? top : m_run;
      const float alpha = __builtin_amdgcn_exp2f(m_run - (m_new == NEG_INF ? 0.0f : m_new));
      m_run = m_new;
      l_run *= alpha;
      e_most = e > e_most ? e : e_most;
      int to = serves(e) ? e_ref : e;
      to = to < e_most - P_REACH ? e_most - P_REACH : to;
      const float by = __builtin_ldexpf(alpha, e_ref - to);
#pragma unroll
      for (int d = 0; d < DT; ++d) acc[d] *= by;
      e_ref = to;
    };
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      // (one branch that is all but never taken)
      if (__builtin_expect((g == 0 && __ballot(top > m_run + P_LAZY) != 0) | !serves(ex[g]), 0)) rescale(ex[g]);
      const float ref = (m_run == NEG_INF ? 0.0f : m_run) - P_SHIFT;
      // (no scale, or one out of reach: at most 2^-100)
      const int de = ex[g] - e_ref < -100 ? -100 : ex[g] - e_ref;
      const float off = ((float)de + lm[g]) - ref;
      float sum[2] = {0.0f, 0.0f};
      h16x8 phi[2], plo[2];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[g][i], f[g], off));
        sum[i & 1] += p;
        phi[i >> 3][i & 7] = (_Float16)p;
        if (F32) plo[i >> 3][i & 7] = (_Float16)(p - (float)phi[i >> 3][i & 7]);
      }
      l_run = __builtin_fmaf(sum[0] + sum[1], __builtin_ldexpf(inv[g], -de), l_run);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const h16x8 va = *reinterpret_cast<const h16x8*>(lds_v[BUF] + (g * 4 + 2 * j + lh) * (D * 16) +
                                                           ((32 * d + li) ^ v_swizzle(2 * j + lh)) * 16);
          acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(va, phi[j], acc[d], 0, 0, 0);
          if (F32) acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(va, plo[j], acc[d], 0, 0, 0);
        }
    }
  };
  for (int tile = tile0; tile < tile_end; tile += 2) {
    step(tile, Index<0>());
    __syncthreads();
    if (tile + 1 < tile_end) {
      step(tile + 1, Index<1>());
      __syncthreads();
    }
  }
  l_run += __shfl_xor(l_run, 32);
  if (32 * wave + li >= rows) return;
  // lane (li, lh) holds channels 32 d + 8 (i / 4) + 4 lh + i % 4 of its row. A
  // row that met no scale above zero keeps e_ref == E_NONE: zeros
  if (vis.used <= 1) {
    const float norm = l_run == 0.0f ? 0.0f : 1.0f / l_run;
    const int64_t at = (int64_t)tok * a.out_stride + (int64_t)qh * D + 4 * lh;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int64_t to = at + 32 * d + 2 * i;
        float o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = __builtin_ldexpf(acc[d][i + k] * norm, e_ref);
        store_heads<SRC>(a.out, to, f32x4{o[0], o[1], o[2], o[3]});
      }
  } else {
    float* part = a.part + (((int64_t)unit * c.n_heads + head) * a.n_splits + split) * P_ROWS * (D + 2);
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<f32x4*>(part + row * D + 32 * d + 2 * i + 4 * lh) =
            f32x4{__builtin_ldexpf(acc[d][i], e_ref), __builtin_ldexpf(acc[d][i + 1], e_ref),
                  __builtin_ldexpf(acc[d][i + 2], e_ref), __builtin_ldexpf(acc[d][i + 3], e_ref)};
    if (lh == 0) {
      part[P_ROWS * D + row] = m_run;
      part[P_ROWS * D + P_ROWS + row] = l_run;
    }
  }
}

// Joins the splits of a unit of UNIT rows: a thread adds four channels of a
// row, eight splits at a time, and everything it needs of them is loaded at
// once.
constexpr int J_THREADS = 256;
constexpr int J_FEW = 8;
constexpr int MAX_SPLITS = 128;

template <int SRC, int D, int UNIT, int NG>
__global__ __launch_bounds__(J_THREADS) void k_attention_join(Cache c, Batch b, Attention a) {
  const int unit = blockIdx.x / c.n_heads, head = blockIdx.x % c.n_heads;
  Span sp;
  const int u = find_unit(b, unit, a.group, UNIT == A_ROWS ? A_SHIFT : P_SHIFT_ROWS, 1, sp);
  const int64_t n_rows = (int64_t)sp.n * a.group;
  const int64_t first_row = (int64_t)u * UNIT;
  if (u < 0 || first_row >= n_rows) return;
  const int rows = (int)(n_rows - first_row < UNIT ? n_rows - first_row : UNIT);
  const Range vis = visible(sp, (int)first_row, rows, a, (int64_t)b.table_width << c.shift, NG);
  const int at = (int)(blockIdx.y * J_THREADS + threadIdx.x);
  const int row = at / (D / 4), ch = at % (D / 4) * 4;
  if (vis.used <= 1 || row >= rows) return;
  constexpr int64_t STEP = (int64_t)UNIT * (D + 2);
  const float* part = a.part + ((int64_t)unit * c.n_heads + head) * a.n_splits * STEP;
  float m = NEG_INF, l = 0.0f;
  f32x4 o = {};
  for (int z0 = 0; z0 < vis.used; z0 += J_FEW) {
    float mz[J_FEW], lz[J_FEW];
    f32x4 oz[J_FEW];
#pragma unroll
    for (int k = 0; k < J_FEW; ++k) {
      const float* pz = part + (z0 + k < vis.used ? z0 + k : z0) * STEP;
      mz[k] = pz[UNIT * D + row];
      lz[k] = pz[UNIT * D + UNIT + row];
      oz[k] = *reinterpret_cast<const f32x4*>(pz + row * D + ch);
    }
    float m_new = m;
#pragma unroll
    for (int k = 0; k < J_FEW; ++k) m_new = __builtin_fmaxf(m_new, mz[k]);   // (repeats change nothing)
    const float ref = m_new == NEG_INF ? 0.0f : m_new;
    const float down = __builtin_amdgcn_exp2f(m - ref);
    m = m_new;
    l *= down;
    o *= down;
#pragma unroll
    for (int k = 0; k < J_FEW; ++k)
      if (z0 + k < vis.used) {
        const float f = __builtin_amdgcn_exp2f(mz[k] - ref);
        l = __builtin_fmaf(lz[k], f, l);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(oz[k][i], f, o[i]);
      }
  }
  const int rr = (int)first_row + row;
  const int64_t to = (int64_t)(sp.row0 + rr / a.group) * a.out_stride + (int64_t)(head * a.group + rr % a.group) * D + ch;
  store_heads<SRC>(a.out, to, l == 0.0f ? f32x4{} : f32x4{o[0] / l, o[1] / l, o[2] / l, o[3] / l});
}

// Many splits of 16 rows (one long sequence): a workgroup per row, each of its
// waves on every fourth split.
// Lane z works out the factor of split z (and z + 64); then every lane adds
// its channels over the splits, whose loads do not wait for each other.
template <int SRC, int D>
__global__ __launch_bounds__(J_THREADS) void k_attention_join_long(Cache c, Batch b, Attention a) {
  constexpr int UNIT = A_ROWS, SHARE = J_THREADS / WAVE;
  constexpr int PER = D / WAVE;   // channels of a lane
  constexpr int BATCH = 8;        // loads in flight
  typedef float f32xp __attribute__((ext_vector_type(PER == 1 ? 2 : PER)));
  __shared__ float share_o[SHARE][D];
  const int unit = blockIdx.x / c.n_heads, head = blockIdx.x % c.n_heads;
  Span sp;
  const int u = find_unit(b, unit, a.group, A_SHIFT, 1, sp);
  const int64_t n_rows = (int64_t)sp.n * a.group;
  const int64_t first_row = (int64_t)u * UNIT;
  if (u < 0 || first_row >= n_rows) return;
  const int rows = (int)(n_rows - first_row < UNIT ? n_rows - first_row : UNIT);
  const Range vis = visible(sp, (int)first_row, rows, a, (int64_t)b.table_width << c.shift, 1);
  const int row = blockIdx.y;
  if (vis.used <= 1 || row >= rows) return;
  const int lane = threadIdx.x & 63, share = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  constexpr int64_t STEP = (int64_t)UNIT * (D + 2);
  const float* part = a.part + ((int64_t)unit * c.n_heads + head) * a.n_splits * STEP;
  float f[2], l = 0.0f, m = NEG_INF;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int z = lane + i * WAVE;
    f[i] = z < vis.used ? part[z * STEP + UNIT * D + row] : NEG_INF;
    m = __builtin_fmaxf(m, f[i]);
  }
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) m = __builtin_fmaxf(m, __shfl_xor(m, s));
  const float ref = m == NEG_INF ? 0.0f : m;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int z = lane + i * WAVE;
    f[i] = __builtin_amdgcn_exp2f(f[i] - ref);
    if (z < vis.used) l = __builtin_fmaf(part[z * STEP + UNIT * D + UNIT + row], f[i], l);
  }
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) l += __shfl_xor(l, s);
  float o[PER] = {};
  for (int z0 = share; z0 < vis.used; z0 += BATCH * SHARE) {
    f32xp v[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int z = z0 + k * SHARE < vis.used ? z0 + k * SHARE : vis.used - 1;
      const float* pz = part + z * STEP + row * D + lane * PER;
      if (PER == 1) v[k][0] = pz[0];
      else v[k] = *reinterpret_cast<const f32xp*>(pz);
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int z = z0 + k * SHARE;
      const float fz = lane_value(z < WAVE ? f[0] : f[1], z & (WAVE - 1));
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (z < vis.used) o[i] = __builtin_fmaf(v[k][i], fz, o[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) share_o[share][lane * PER + i] = o[i];
  __syncthreads();
  if (share > 0) return;
#pragma unroll
  for (int w = 1; w < SHARE; ++w)
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] += share_o[w][lane * PER + i];
  const int rr = (int)first_row + row;
  const int64_t at = (int64_t)(sp.row0 + rr / a.group) * a.out_stride + (int64_t)(head * a.group + rr % a.group) * D + lane * PER;
#pragma unroll
  for (int k = 0; k < PER; ++k) store_at<SRC>(a.out, at + k, l == 0.0f ? 0.0f : o[k] / l);
}

template <int SRC, int D, int UNIT, int NG>
void launch_join(const Cache& c, const Batch& b, const Attention& a, uint32_t blocks, hipStream_t s) {
  if (UNIT == A_ROWS && a.n_splits > J_FEW)
    hipLaunchKernelGGL((k_attention_join_long<SRC, D>), dim3(blocks, A_ROWS), dim3(J_THREADS), 0, s, c, b, a);
  else
    hipLaunchKernelGGL((k_attention_join<SRC, D, UNIT, NG>), dim3(blocks, (UNIT * D / 4 + J_THREADS - 1) / J_THREADS),
                       dim3(J_THREADS), 0, s, c, b, a);
}

// ---------------------------------------------------------------------------
// host side

bool valid_cache(const qr_kv8* c) {
  return c && c->n_blocks >= 0 && c->n_blocks <= INT32_MAX && c->n_heads >= 1 && c->n_heads <= MAX_HEADS &&
         (c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256) &&
         (c->block_tokens == 32 || c->block_tokens == 64 || c->block_tokens == 128);
}

int check_batch(const qr_kv8* c, int dtype, int64_t n_tok, int64_t n_seq, int64_t table_width) {
  if (dtype != QR_F32 && dtype != QR_BF16) return qr_fail(QR_EINVAL_TYPE, "element type %d is not QR_F32 or QR_BF16", dtype);
  if (!valid_cache(c))
    return qr_fail(QR_EINVAL_SHAPE, "the cache needs 0 <= n_blocks < 2^31, 1 <= n_heads <= %d, head_dim 64, 128 or 256 "
                   "and block_tokens 32, 64 or 128", MAX_HEADS);
  if (n_tok < 0 || n_seq < 0 || table_width < 0)
    return qr_fail(QR_EINVAL_SHAPE, "negative n_tok, n_seq or table_width");
  if (n_tok > INT32_MAX || n_seq > INT32_MAX - 1 || table_width > INT32_MAX)
    return qr_fail(QR_EOVERFLOW, "n_tok, n_seq and table_width must be below 2^31");
  return QR_OK;
}

int check_stride(const char* what, int64_t stride, int64_t least, int64_t n_tok) {
  if (stride < least || stride % 8 != 0)
    return qr_fail(QR_EINVAL_SHAPE, "%s=%lld must be a multiple of 8, at least %lld", what, (long long)stride,
                   (long long)least);
  if (n_tok > 0 && stride > INT64_MAX / 4 / n_tok) return qr_fail(QR_EOVERFLOW, "%s too large", what);
  return QR_OK;
}

int check_pointers(const qr_kv8* c, const int32_t* cu, const int32_t* kv_len, const int32_t* table, int64_t table_width) {
  if (!cu || !kv_len || (!table && table_width > 0)) return qr_fail(QR_EINVAL_PTR, "cu, kv_len and table must be non-NULL");
  if (!qr_aligned(cu, 4) || !qr_aligned(kv_len, 4) || !qr_aligned(table, 4))
    return qr_fail(QR_EINVAL_PTR, "cu, kv_len and table must be 4-byte aligned");
  if (c->n_blocks > 0 && (!c->k || !c->v || !c->kd || !c->vd)) return qr_fail(QR_EINVAL_PTR, "the cache's arrays must be non-NULL");
  if (!qr_aligned(c->k, 16) || !qr_aligned(c->v, 16) || !qr_aligned(c->kd, 4) || !qr_aligned(c->vd, 4))
    return qr_fail(QR_EINVAL_PTR, "the cache's codes must be 16-byte aligned, its scales 4-byte aligned");
  return QR_OK;
}

Cache device_cache(const qr_kv8* c) {
  return {c->k, c->v, c->kd, c->vd, (int)c->n_blocks, (int)c->n_heads, c->block_tokens == 32 ? 5 : c->block_tokens == 64 ? 6 : 7};
}

// Units of a call that takes one piece of a block at a time.
int64_t piece_units(const qr_kv8* c, int64_t n_tok, int64_t n_seq) { return n_tok / c->block_tokens + 2 * n_seq; }

// How a call of attention is cut: units of 16 or 128 rows, and splits of the
// tokens where that leaves CUs without work. The rules go by what the host
// knows, the table's width and averages over the sequences: a table much wider
// than its sequences costs short ones a second launch, one long sequence among
// many short ones is split as little as they are, and prompts mixed with
// single tokens take one kernel for both.
struct Cut {
  bool many;        // the kernel for many rows
  int64_t units, splits;
};

Cut cut_for(const qr_kv8* c, int64_t n_tok, int64_t n_seq, int64_t group, int64_t table_width) {
  Cut k;
  const int64_t rows = (n_tok * group + n_seq - 1) / n_seq;   // of a sequence, on average
  // two units of 16 rows read the tokens twice and still win (64 sequences of
  // 1000 tokens, 32 rows each: 39 against 46 us); three do not (48 rows: 59
  // against 51 us, 8 sequences of 2000: 30 against 24 us)
  k.many = rows > 2 * A_ROWS;
  const int64_t unit = k.many ? P_ROWS : A_ROWS;
  k.units = n_tok * group / unit + n_seq;
  const int64_t busy = n_seq * ((rows + unit - 1) / unit) * c->n_heads;
  const int64_t groups = table_width * (c->block_tokens / GROUP);
  // up to 1024 tokens one launch: 10.2 us for 700 tokens of 4 sequences,
  // against 6.9 and 2.5 us and what lies between two launches
  const int64_t most = !k.many && groups <= 32 ? 1 : (groups + A_MIN_GROUPS - 1) / A_MIN_GROUPS;
  const int64_t want = k.many ? 512 : 2048;   // workgroups: two, eight per CU
  k.splits = (want + busy - 1) / busy;
  if (k.splits > most) k.splits = most;
  if (k.splits > MAX_SPLITS) k.splits = MAX_SPLITS;
  if (k.splits < 1) k.splits = 1;
  return k;
}

template <int SRC, int D>
int launch_attention(const Cache& c, const Batch& b, const Attention& a, const Cut& k, hipStream_t s) {
  constexpr int NG = D == 256 ? 1 : 2;   // what two LDS buffers hold in 64 KB
  const uint32_t blocks = (uint32_t)(k.units * c.n_heads);
  const dim3 grid(blocks, (uint32_t)a.n_splits);
  if (k.many) hipLaunchKernelGGL((k_attention_kv8_rows<SRC, D, NG>), grid, dim3(P_WAVES * WAVE), 0, s, c, b, a);
  else hipLaunchKernelGGL((k_attention_kv8<SRC, D>), grid, dim3(A_WAVES * WAVE), 0, s, c, b, a);
  if (a.n_splits > 1) {
    const int rc = qr_check_launch("k_attention_kv8");
    if (rc != QR_OK) return rc;
    if (k.many) launch_join<SRC, D, P_ROWS, NG>(c, b, a, blocks, s);
    else launch_join<SRC, D, A_ROWS, 1>(c, b, a, blocks, s);
  }
  return qr_check_launch("k_attention_kv8");
}

template <int SRC, int D>
int launch_append(const Cache& c, const Batch& b, const void* k, const void* v, int64_t ks, int64_t vs, uint32_t units,
                  hipStream_t s) {
  const int block = 1 << c.shift, threads = rw_threads<D>(block);
  const dim3 grid(units * (uint32_t)c.n_heads, 2);
  if (squares_of<D>(block) > threads)   // 128 tokens of 256 channels
    hipLaunchKernelGGL((k_kv8_append<SRC, D, D == 256 ? 2 : 1>), grid, dim3(threads), 0, s, c, b, k, v, ks, vs);
  else
    hipLaunchKernelGGL((k_kv8_append<SRC, D, 1>), grid, dim3(threads), 0, s, c, b, k, v, ks, vs);
  return qr_check_launch("k_kv8_append");
}

template <int DST, int D>
int launch_read(const Cache& c, const Batch& b, void* k, void* v, int64_t ks, int64_t vs, uint32_t units, hipStream_t s) {
  hipLaunchKernelGGL((k_kv8_read<DST, D>), dim3(units * (uint32_t)c.n_heads, 2), dim3(rw_threads<D>(1 << c.shift)), 0, s,
                     c, b, k, v, ks, vs);
  return qr_check_launch("k_kv8_read");
}

// The checks that writing and reading share; QR_OK with *units == 0: nothing to do.
int check_rows(const qr_kv8* c, int dtype, const void* k, const void* v, int64_t k_stride, int64_t v_stride,
               int64_t n_tok, int64_t n_seq, const int32_t* cu, const int32_t* kv_len, const int32_t* table,
               int64_t table_width, int64_t* units) {
  *units = 0;
  int rc = check_batch(c, dtype, n_tok, n_seq, table_width);
  if (rc == QR_OK) rc = check_stride("k_stride", k_stride, c->n_heads * c->head_dim, n_tok);
  if (rc == QR_OK) rc = check_stride("v_stride", v_stride, c->n_heads * c->head_dim, n_tok);
  if (rc != QR_OK || n_tok == 0 || n_seq == 0) return rc;
  rc = check_pointers(c, cu, kv_len, table, table_width);
  if (rc != QR_OK) return rc;
  if (!k || !v || !qr_aligned(k, 16) || !qr_aligned(v, 16))
    return qr_fail(QR_EINVAL_PTR, "k and v must be non-NULL and 16-byte aligned");
  *units = piece_units(c, n_tok, n_seq);
  if (*units * c->n_heads > UINT32_MAX / RW_THREADS) return qr_fail(QR_EOVERFLOW, "n_tok and n_seq need too many workgroups for one launch");
  return QR_OK;
}

}  // namespace

extern "C" {

size_t qr_kv8_code_bytes(const qr_kv8* c) {
  if (!valid_cache(c)) return 0;
  return (size_t)(c->n_blocks * c->n_heads * c->block_tokens * c->head_dim);
}

int qr_kv8_append(const qr_kv8* c, int src, const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                  int64_t n_tok, int64_t n_seq, const int32_t* cu, const int32_t* kv_len, const int32_t* table,
                  int64_t table_width, void* stream) {
  qr_clear_error();
  int64_t units;
  const int rc = check_rows(c, src, k, v, k_stride, v_stride, n_tok, n_seq, cu, kv_len, table, table_width, &units);
  if (rc != QR_OK || units == 0) return rc;
  const Cache cc = device_cache(c);
  const Batch b = {cu, kv_len, table, (int)table_width, (int)n_seq, (int)n_tok};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const uint32_t n = (uint32_t)units;
  switch (c->head_dim) {
    case 64: return src == QR_BF16 ? launch_append<QR_BF16, 64>(cc, b, k, v, k_stride, v_stride, n, s)
                                   : launch_append<QR_F32, 64>(cc, b, k, v, k_stride, v_stride, n, s);
    case 128: return src == QR_BF16 ? launch_append<QR_BF16, 128>(cc, b, k, v, k_stride, v_stride, n, s)
                                    : launch_append<QR_F32, 128>(cc, b, k, v, k_stride, v_stride, n, s);
    default: return src == QR_BF16 ? launch_append<QR_BF16, 256>(cc, b, k, v, k_stride, v_stride, n, s)
                                   : launch_append<QR_F32, 256>(cc, b, k, v, k_stride, v_stride, n, s);
  }
}

int qr_kv8_read(const qr_kv8* c, int dst, void* k, void* v, int64_t k_stride, int64_t v_stride, int64_t n_tok,
                int64_t n_seq, const int32_t* cu, const int32_t* kv_len, const int32_t* table, int64_t table_width,
                void* stream) {
  qr_clear_error();
  int64_t units;
  const int rc = check_rows(c, dst, k, v, k_stride, v_stride, n_tok, n_seq, cu, kv_len, table, table_width, &units);
  if (rc != QR_OK || units == 0) return rc;
  const int64_t esize = dst == QR_BF16 ? 2 : 4;
  if (serve::rows_meet(k, k_stride * esize, v, v_stride * esize, c->n_heads * c->head_dim * esize, n_tok))
    return qr_fail(QR_EINVAL_PTR, "k and v must not overlap");
  const Cache cc = device_cache(c);
  const Batch b = {cu, kv_len, table, (int)table_width, (int)n_seq, (int)n_tok};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const uint32_t n = (uint32_t)units;
  switch (c->head_dim) {
    case 64: return dst == QR_BF16 ? launch_read<QR_BF16, 64>(cc, b, k, v, k_stride, v_stride, n, s)
                                   : launch_read<QR_F32, 64>(cc, b, k, v, k_stride, v_stride, n, s);
    case 128: return dst == QR_BF16 ? launch_read<QR_BF16, 128>(cc, b, k, v, k_stride, v_stride, n, s)
                                    : launch_read<QR_F32, 128>(cc, b, k, v, k_stride, v_stride, n, s);
    default: return dst == QR_BF16 ? launch_read<QR_BF16, 256>(cc, b, k, v, k_stride, v_stride, n, s)
                                   : launch_read<QR_F32, 256>(cc, b, k, v, k_stride, v_stride, n, s);
  }
}

size_t qr_attention_kv8_workspace_bytes(const qr_kv8* c, int64_t n_q_heads, int64_t n_tok, int64_t n_seq,
                                        int64_t table_width) {
  if (!valid_cache(c) || n_q_heads <= 0 || n_q_heads % c->n_heads != 0 || n_tok <= 0 || n_seq <= 0 || table_width < 0 ||
      n_tok > INT32_MAX || n_seq > INT32_MAX - 1 || table_width > INT32_MAX || n_q_heads / c->n_heads > 1024 ||
      n_tok * n_q_heads > INT32_MAX)
    return 0;
  const int64_t group = n_q_heads / c->n_heads;
  const Cut k = cut_for(c, n_tok, n_seq, group, table_width);
  if (k.splits == 1) return 0;
  return (size_t)(k.units * c->n_heads * k.splits * (k.many ? P_ROWS : A_ROWS) * (c->head_dim + 2)) * sizeof(float);
}

int qr_attention_kv8(const qr_kv8* c, int src, const void* q, int64_t q_stride, int64_t n_q_heads, int64_t n_tok,
                     int64_t n_seq, const int32_t* cu, const int32_t* kv_len, const int32_t* table, int64_t table_width,
                     float scale, int64_t window, void* out, int64_t out_stride, void* workspace,
                     size_t workspace_bytes, void* stream) {
  qr_clear_error();
  int rc = check_batch(c, src, n_tok, n_seq, table_width);
  if (rc != QR_OK) return rc;
  if (n_q_heads <= 0 || n_q_heads % c->n_heads != 0 || n_q_heads / c->n_heads > 1024)
    return qr_fail(QR_EINVAL_SHAPE, "n_q_heads=%lld must be a multiple of n_heads=%lld, at most 1024 times it",
                   (long long)n_q_heads, (long long)c->n_heads);
  if (window < 0 || !(scale - scale == 0.0f)) return qr_fail(QR_EINVAL_SHAPE, "window must not be negative, scale must be finite");
  rc = check_stride("q_stride", q_stride, n_q_heads * c->head_dim, n_tok);
  if (rc == QR_OK) rc = check_stride("out_stride", out_stride, n_q_heads * c->head_dim, n_tok);
  if (rc != QR_OK || n_tok == 0 || n_seq == 0) return rc;
  if (n_tok * n_q_heads > INT32_MAX) return qr_fail(QR_EOVERFLOW, "n_tok * n_q_heads must be below 2^31");
  rc = check_pointers(c, cu, kv_len, table, table_width);
  if (rc != QR_OK) return rc;
  if (!q || !out || !qr_aligned(q, 16) || !qr_aligned(out, 16))
    return qr_fail(QR_EINVAL_PTR, "q and out must be non-NULL and 16-byte aligned");
  const int64_t group = n_q_heads / c->n_heads;
  const Cut cut = cut_for(c, n_tok, n_seq, group, table_width);
  if (cut.units * c->n_heads > UINT32_MAX / 256) return qr_fail(QR_EOVERFLOW, "n_tok and n_seq need too many workgroups for one launch");
  const size_t need = qr_attention_kv8_workspace_bytes(c, n_q_heads, n_tok, n_seq, table_width);
  if (need > 0 && (!workspace || !qr_aligned(workspace, 256)))
    return qr_fail(QR_EINVAL_PTR, "workspace must be non-NULL and 256-byte aligned");
  if (workspace_bytes < need)
    return qr_fail(QR_EINVAL_SHAPE, "workspace has %zu bytes, %zu are needed", workspace_bytes, need);
  const int64_t esize = src == QR_BF16 ? 2 : 4;
  if (serve::rows_meet(q, q_stride * esize, out, out_stride * esize, n_q_heads * c->head_dim * esize, n_tok))
    return qr_fail(QR_EINVAL_PTR, "q and out must not overlap");
  const Cache cc = device_cache(c);
  const Batch b = {cu, kv_len, table, (int)table_width, (int)n_seq, (int)n_tok};
  const Attention a = {q, out, reinterpret_cast<float*>(workspace), q_stride, out_stride, scale * 1.44269504088896340736f,
                       window < (int64_t)1 << 32 ? window : (int64_t)1 << 32, (int)group, (int)cut.splits, (int)cut.units};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  switch (c->head_dim) {
    case 64: return src == QR_BF16 ? launch_attention<QR_BF16, 64>(cc, b, a, cut, s) : launch_attention<QR_F32, 64>(cc, b, a, cut, s);
    case 128: return src == QR_BF16 ? launch_attention<QR_BF16, 128>(cc, b, a, cut, s) : launch_attention<QR_F32, 128>(cc, b, a, cut, s);
    default: return src == QR_BF16 ? launch_attention<QR_BF16, 256>(cc, b, a, cut, s) : launch_attention<QR_F32, 256>(cc, b, a, cut, s);
  }
}

}  // extern "C"
