// serve_internal.h -- what the serving translation units of libqrow.so share
// (not part of the C-ABI).
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "qrow.h"
#include "serve/qrow_i8.h"

namespace serve {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
// Vectors at any element of the caller's rows, whose strides are free: memory
// instructions take them unaligned.
typedef uint16_t u16x8_any __attribute__((ext_vector_type(8), aligned(2)));
typedef uint16_t u16x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));

constexpr int WAVE = 64;

__device__ __forceinline__ float bf16_value(uint16_t h) { return __builtin_bit_cast(float, (uint32_t)h << 16); }

// fp32 to bf16, round to nearest even (NaN stays NaN).
__device__ __forceinline__ uint16_t bf16_bits(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// What a wave's lanes wrote to LDS is there for its other lanes.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Operands are loaded from buffers: a base and a step in scalar registers, a
// lane's place in one 32-bit register that never changes (64-bit addresses, and
// the registers they were made in, had loads wait for the ones before).
typedef __amdgpu_buffer_rsrc_t Buffer;

__device__ __forceinline__ Buffer buffer_of(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00027000);
}

// A place behind every buffer: such a lane gets zeros and asks for nothing.
constexpr uint32_t NOWHERE = 0x80000000u;

__device__ __forceinline__ i32x4 load16(Buffer b, uint32_t lane_at, uint32_t at) {
  return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(b, lane_at, at, 0));
}

// Weights are read once: loads that leave no trace in the caches, of whole
// 128-byte lines (eight rows a wave's instruction). They pass at 7.0 TB/s, the
// same lines in halves, 16 rows at a time as the matrix instruction takes them,
// at 6.0, and both at 6.3 through the caches (3.8 GB, nothing else done).
__device__ __forceinline__ i32x4 load16_once(Buffer b, uint32_t lane_at, uint32_t at) {
  constexpr int NONTEMPORAL = 2;
  return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(b, lane_at, at, NONTEMPORAL));
}

// multiply(stage, k) for k = from, from + step, ... below to, with the loads
// DEPTH stages ahead: every stage is asked for again as soon as it is used.
template <int DEPTH, typename Stage, typename Load, typename Multiply>
__device__ __forceinline__ void pipeline(int from, int to, int step, Load load, Multiply multiply) {
  Stage stage[DEPTH];
#pragma unroll
  for (int s = 0; s < DEPTH; ++s)
    if (from + s * step < to) load(stage[s], from + s * step);
  int k = from;
  for (; k + (2 * DEPTH - 1) * step < to; k += DEPTH * step) {
#pragma unroll
    for (int s = 0; s < DEPTH; ++s) {
      multiply(stage[s], k + s * step);
      load(stage[s], k + (s + DEPTH) * step);
      __builtin_amdgcn_sched_barrier(0);   // or the loads of all stages are waited for together
    }
  }
  for (; k < to; k += DEPTH * step) {
#pragma unroll
    for (int s = 0; s < DEPTH; ++s) {
      if (k + s * step < to) multiply(stage[s], k + s * step);
      if (k + (s + DEPTH) * step < to) load(stage[s], k + (s + DEPTH) * step);
    }
  }
}

// 128 bytes of 16 rows: `low` has rows 0-7, `high` rows 8-15, lanes li < 8 of
// each their first 64 bytes, the others their last. As the matrix instruction
// takes them (row li, bytes 16 lk): the first halves into `low`, the last ones
// into `high`, by a turn of half the lanes of each.
__device__ __forceinline__ void turn(i32x4& low, i32x4& high) {
  constexpr int ROR8 = 0x128;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int a = low[i], b = high[i];
    low[i] = __builtin_amdgcn_update_dpp(a, b, ROR8, 0xf, 0xc, false);
    high[i] = __builtin_amdgcn_update_dpp(b, a, ROR8, 0xf, 0x3, false);
  }
}

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

// Eight values rounded to codes, in eight bytes. A sum with 1.5 * 2^23 is
// rounded to a whole number, to even like rint, and has it in its low bits.
__device__ __forceinline__ u32x2 pack_codes(const float (&v)[8], float inv) {
  u32x2 o;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = __builtin_bit_cast(uint32_t, v[4 * w + i] * inv + 0x1.8p23f);
    // bytes 0 of two words each side by side, then the two halves
    const uint32_t lo = __builtin_amdgcn_perm(u[1], u[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(u[3], u[2], 0x04000c0cu);
    o[w] = lo | hi;
  }
  return o;
}

// The scale of codes whose largest magnitude has the bits `top`, and the
// factor that makes the codes: zero where there are none to make.
struct CodeScale {
  float d, inv;
  bool finite;
};

__device__ __forceinline__ CodeScale code_scale(uint32_t top) {
  const float amax = __builtin_bit_cast(float, top);
  CodeScale s = {amax / 127.0f, 127.0f / amax, top < 0x7f800000u};
  if (!s.finite || !(s.inv < __builtin_inff())) {
    s.inv = 0.0f;
    s.d = s.finite ? 0.0f : __builtin_nanf("");
  }
  return s;
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

// x / (1 + exp(t)) in fp32. The hardware's exp2 and reciprocal are good to a
// last place each; the bits that t log2(e) loses are carried on (they count
// |t| times), and one step mends the quotient. Some 14 instructions; the exact
// division and exp of the math library take three times that.
__device__ __forceinline__ float over_one_plus_exp(float x, float t) {
  const float hi = t * 1.44269502162933349609375f;
  const float lo = __builtin_fmaf(t, 1.92596299112661746887e-8f, __builtin_fmaf(t, 1.44269502162933349609375f, -hi));
  const float p = __builtin_amdgcn_exp2f(hi);
  const float d = 1.0f + __builtin_fmaf(p, lo * 0.693147180559945309417f, p);
  const float r = __builtin_amdgcn_rcpf(d);
  const float q = x * r;
  // (beyond, exp(t) is no number any more, and what is left of x subnormal)
  return t > 88.0f ? x * 0.0f : t < -88.0f ? x : __builtin_fmaf(__builtin_fmaf(-d, q, x), r, q);
}
__device__ __forceinline__ double over_one_plus_exp(double x, double t) { return x / (1.0 + exp(t)); }

// Activations (QR_ACT_*). GELU is x times half erfc(-x / sqrt 2): one plus erf
// would lose the bits of what is left of it at negative x. Its tanh form is
// x / (1 + exp(-2u)), since (1 + tanh u) / 2 = 1 / (1 + exp(-2u)).
template <typename T>
__device__ __forceinline__ T activation(int act, T x) {
  switch (act) {
    case QR_ACT_RELU: return x > T(0) || x != x ? x : T(0);
    case QR_ACT_SILU: return over_one_plus_exp(x, -x);
    case QR_ACT_GELU: return x * (T(0.5) * erfc(x * T(-0.70710678118654752440)));
    case QR_ACT_GELU_TANH:
      return over_one_plus_exp(x, x * (T(-1.59576912160573071176) - T(0.07135481627260025) * x * x));
    default: return x;
  }
}

// The same of N values with one branch: their steps then run side by side
// (8192 tokens, 11008 x 4096 gated: one by one 862 us, four 839, eight 797 to 837).
template <int N>
__device__ __forceinline__ void activate(int act, float (&v)[N]) {
  const auto each = [&](int kind) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = activation(kind, v[i]);
  };
  switch (act) {
    case QR_ACT_RELU: each(QR_ACT_RELU); break;
    case QR_ACT_SILU: each(QR_ACT_SILU); break;
    case QR_ACT_GELU: each(QR_ACT_GELU); break;
    case QR_ACT_GELU_TANH: each(QR_ACT_GELU_TANH); break;
    default: break;
  }
}

// Whether any of n rows of `row` bytes, a_step bytes apart, shares memory with
// one of the rows at b: parts of one buffer lie between each other without
// meeting.
inline bool rows_meet(const void* a_ptr, int64_t a_step, const void* b_ptr, int64_t b_step, int64_t row, int64_t n) {
  uintptr_t a = (uintptr_t)a_ptr, b = (uintptr_t)b_ptr;
  if (a + (uintptr_t)((n - 1) * a_step + row) <= b || b + (uintptr_t)((n - 1) * b_step + row) <= a) return false;
  if (a_step == b_step) {
    const int64_t apart = (int64_t)((a < b ? b - a : a - b) % (uintptr_t)a_step);
    return apart < row || a_step - apart < row;
  }
  for (int64_t i = 0, j = 0; i < n && j < n;) {   // both ascend: the one that ends first goes on
    if (a + row <= b) a += a_step, ++i;
    else if (b + row <= a) b += b_step, ++j;
    else return true;
  }
  return false;
}

// Whether the n rows of `row` bytes at a, a_step bytes apart, share memory with
// the `bytes` bytes at b.
inline bool rows_meet_range(const void* a_ptr, int64_t a_step, int64_t row, int64_t n, const void* b_ptr,
                            int64_t bytes) {
  const uintptr_t a = (uintptr_t)a_ptr, b = (uintptr_t)b_ptr, e = b + (uintptr_t)bytes;
  if (n == 0 || bytes == 0 || e <= a || a + (uintptr_t)((n - 1) * a_step + row) <= b) return false;
  if (b <= a) return true;                            // reaches into the first row
  const int64_t into = (int64_t)((b - a) % (uintptr_t)a_step);
  return into < row || (int64_t)(e - b) > a_step - into;   // (a row follows: the range starts before the last one's end)
}

}  // namespace serve
