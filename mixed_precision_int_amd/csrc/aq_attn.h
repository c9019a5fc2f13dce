// Attention over the 4-bit cache: device helpers that the kernel for few rows
// and the kernel for prompts share.
//
// Arithmetic.  A cached feature is s (c - z) with s of its token: c - z is a
// whole number of -15 .. 15, exact in FP16, and s stays outside the products.
// Products run on the FP16 matrix instructions with FP32 sums; q and the
// weights, which are FP32, enter as two FP16 pieces, high and low, 22 bits:
//  * q' = q * 2^(13 - E), E the exponent of its row's largest value, so that
//    every piece is in FP16's range whatever the row's magnitude (power-of-two
//    factors are exact);
//  * the weight of token t in the value sum, p_t s_t, is formed as
//    2^(a_t - M) f_t, a_t = score + e_t in powers of two, s_t = f_t 2^e_t with f_t
//    in [1, 2), and M the running maximum of a: at most 2 whatever the scales of
//    the values are.  The softmax's denominator takes 2^(a_t - M) 2^(-e_t).
// So the output is sum 2^(a-M) f (c - z) over sum 2^(a-M) 2^-e, and neither
// overflows.
//
// A word that holds NaN (a vector that was not finite): the key's NaN goes
// through the score; the value's 2^-e comes out as -infinity, which the
// denominator keeps, and a negative or NaN denominator ends as NaN.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "aq_layer.h"

namespace aq {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ h2 as_h2(uint32_t x) { return __builtin_bit_cast(h2, x); }

constexpr float kNone = -3.402823466e38f;  // the running maximum before the first key
constexpr uint32_t kPieceBias = 13;        // weights and q are held times 2^13

// ---- codes to FP16
// 0x6400 | c is 1024 + c in FP16 and 0x6400 | 16 c is 1024 + 16 c, both exact, so
// that a nibble widens by one and-or and one packed operation that also takes
// z off: (1024 + c) - (1024 + z), and (1024 + 16 c) / 16 - (64 + z).
// The two negated constants for zero points z0 (low half) and z1.
struct Zero { h2 lo, hi; };
__device__ __forceinline__ Zero zero_of(uint32_t z0, uint32_t z1) {
  const uint32_t z = z0 | z1 << 16;
  return Zero{as_h2(0xE400E400u | z), as_h2(0xD400D400u | z << 4)};
}
__device__ __forceinline__ h2 widen_lo(uint32_t x, const Zero &z) { return as_h2((x & 0x000F000Fu) | 0x64006400u) + z.lo; }
__device__ __forceinline__ h2 widen_hi(uint32_t x, const Zero &z) {
  const h2 sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
  return as_h2((x & 0x00F000F0u) | 0x64006400u) * sixteenth + z.hi;
}
// A word of 8 features of one token, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ h8 widen8(uint32_t w, const Zero &z) {
  const h2 a = widen_lo(w, z), b = widen_hi(w, z), c = widen_lo(w >> 8, z), d = widen_hi(w >> 8, z);
  return h8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// ---- words
__device__ __forceinline__ float scale_of(uint32_t w) { return __uint_as_float(w & ~15u); }
// s = f 2^e: f * 2^13 (for the weight's pieces), e, and 2^-e (-infinity for NaN).
__device__ __forceinline__ float frac_of(uint32_t w) {
  return __uint_as_float((w & 0x007FFFF0u) | (127u + kPieceBias) << 23);
}
__device__ __forceinline__ float exp_of(uint32_t w) { return (float)((int)(w >> 23 & 255u) - 127); }
__device__ __forceinline__ float inv_exp_of(uint32_t w) {
  return __uint_as_float((uint32_t)(254 - (int)(w >> 23 & 255u)) << 23);
}

// ---- pieces
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
// The factor 2^(13 - E) for a row whose largest finite magnitude is amax, and
// its inverse; at most 2^126, so that both are normal.
__device__ __forceinline__ void row_factor(float amax, float &up, float &down) {
  const int f = min(267 - (int)(__float_as_uint(amax) >> 23), 253);
  up = __uint_as_float((uint32_t)f << 23);
  down = __uint_as_float((uint32_t)(254 - f) << 23);
}
__device__ __forceinline__ void pieces(float x, _Float16 &hi, _Float16 &lo) {
  hi = (_Float16)x;
  lo = (_Float16)(x - (float)hi);
}
// |x| where it is finite, else 0.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}
// Eight features of a row in widen8's order.
__device__ __forceinline__ void pieces8(const float (&x)[8], float up, h8 &hi, h8 &lo) {
  constexpr int order[8] = {0, 4, 1, 5, 2, 6, 3, 7};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    _Float16 a, b;
    pieces(x[order[j]] * up, a, b);
    hi[j] = a;
    lo[j] = b;
  }
}

// 1 / denominator: no key gives zeros, a key or value that was not finite NaN.
__device__ __forceinline__ float inv_sum(float l) {
  return l > 0.f ? 1.f / l : l == 0.f ? 0.f : __uint_as_float(0x7FC00000u);
}

// ---- rows
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
// Row tile `tile` of T rows: its sequence, first row, rows of the sequence,
// first token's row of q, and tokens and cached tokens of the sequence.  Called
// by whole waves; false where no such tile exists.
struct Rows { int b, r0, rows, first, n, len; };
template <int T>
__device__ __forceinline__ bool find_rows(const AttnArgs &a, int tile, Rows &r) {
  const int most = a.width << a.c.shift;
  if (!a.cu) {
    const int per = (a.G + T - 1) / T;
    r.b = tile / per;
    r.r0 = (tile - r.b * per) * T;
    r.first = r.b;
    r.n = 1;
  } else {
    // tiles of 64 sequences at a time, summed over the wave
    const int lane = threadIdx.x & 63;
    int left = tile, b0 = 0;
    for (;; b0 += 64) {
      if (b0 >= a.B) return false;
      const int b = b0 + lane;
      int lo = 0, n = 0;
      if (b < a.B) {
        lo = min(max(a.cu[b], 0), a.M);
        n = min(max(a.cu[b + 1], lo), a.M) - lo;
      }
      const int t = (int)(((long long)n * a.G + T - 1) / T);
      int upto = t;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(upto, o);
        if (lane >= o) upto += v;
      }
      const uint64_t past = __ballot(upto > left);
      if (past) {
        const int l = __ffsll((unsigned long long)past) - 1;
        r.b = b0 + l;
        r.r0 = (left - (__shfl(upto, l) - __shfl(t, l))) * T;
        r.first = __shfl(lo, l);
        r.n = __shfl(n, l);
        break;
      }
      left -= __shfl(upto, 63);
    }
  }
  // (uniform over the wave, which the compiler does not see)
  r.b = uniform(r.b);
  r.r0 = uniform(r.r0);
  r.first = uniform(r.first);
  r.n = uniform(r.n);
  r.rows = r.n * a.G;
  r.len = uniform(min(max(a.kv_len[r.b], 0), most));
  return true;
}

// ---- keys
// The range of key units of a split: [u0, u1) and the ranges there are.
struct Range { int u0, u1, ranges; };
__device__ __forceinline__ Range split_range(int limit, int unit, int splits, int split) {
  const int units = (limit + unit - 1) / unit;
  const int per = max(1, (units + splits - 1) / splits);
  Range r;
  r.ranges = max(1, (units + per - 1) / per);
  r.u0 = min(units, split * per);
  r.u1 = min(units, r.u0 + per);
  return r;
}

}  // namespace aq
