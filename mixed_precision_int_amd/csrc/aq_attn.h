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
//    in [1, 2), and M about the running maximum of a: bounded whatever the scales of
//    the values are.  The softmax's denominator takes 2^(a_t - M) 2^(-e_t).
// So the output is sum 2^(a-M) f (c - z) over sum 2^(a-M) 2^-e.  Scales lie below 2^64, and those below
// 2^-48 keep e = -48 and a smaller f (the append's are 2^-40 at least): beside a value of any other scale a
// token's weight is then above FP32's least down to a softmax weight of 2^-20, and stays in the
// denominator.
//
// (log2(s) in the place of e and no f is a multiplication less for each score, 574 against 590 us for a
// prompt of 6000 tokens; but a scale below the least counts as that then, not as what it is.)
//
// A word of 2^64 or more, negative or NaN (a vector that was not finite) is NaN: the key's goes
// through the score, the value's through the weight, and no further than the rows that see it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "aq_kv4.h"
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
// M follows the scores only where one exceeds it by 2^kSlack (the rescaling of the sums is half of
// the softmax's work where it follows each), and stands 2^kLift below what it follows: weights are at
// most 2 * 2^(kSlack + kLift), below FP16's largest, and their pieces keep 22 bits down to 2^-7 of the
// maximum and 2^-29 of it in absolute terms.
constexpr float kSlack = 8.f, kLift = 5.f;

__device__ __forceinline__ h8 join8(h2 a, h2 b, h2 c, h2 d) { return h8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y}; }

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
// The nibbles' masks in vector registers: an instruction takes one scalar constant, and an
// and-or has two.
struct Masks { uint32_t lo, hi; };
__device__ __forceinline__ Masks masks() {
  Masks m = {0x000F000Fu, 0x00F000F0u};
  asm volatile("" : "+v"(m.lo), "+v"(m.hi));
  return m;
}
__device__ __forceinline__ h2 widen_lo(uint32_t x, const Masks &m, const Zero &z) { return as_h2((x & m.lo) | 0x64006400u) + z.lo; }
__device__ __forceinline__ h2 widen_hi(uint32_t x, const Masks &m, const Zero &z) {
  const h2 sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
  return __builtin_elementwise_fma(as_h2((x & m.hi) | 0x64006400u), sixteenth, z.hi);
}
// A word of 8 features of one token, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ h8 widen8(uint32_t w, const Masks &m, const Zero &z) {
  return join8(widen_lo(w, m, z), widen_hi(w, m, z), widen_lo(w >> 8, m, z), widen_hi(w >> 8, m, z));
}


// ---- words
__device__ __forceinline__ float scale_of(uint32_t w) { return scale_held(w); }
// e of s = f 2^e, as FP32, and 2^-e.
__device__ __forceinline__ void exponent_of(uint32_t w, float &e, float &inv) {
  const int E = min(max((int)(w >> 23 & 255u), 79), 191);
  e = (float)(E - 127);
  inv = __uint_as_float((uint32_t)(254 - E) << 23);
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
// Maximum over lanes n, n ^ 16, n ^ 32 and n ^ 48; over n and n ^ 32.
__device__ __forceinline__ float max_half(float x) {
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}
__device__ __forceinline__ float max_halves(float x) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return max_half(fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1])));
}
__device__ __forceinline__ uint32_t max_halves(uint32_t x) {
  const auto p = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  const uint32_t m = max(p[0], p[1]);
  const auto q = __builtin_amdgcn_permlane32_swap(m, m, false, false);
  return max(q[0], q[1]);
}
// Sum over lanes n, n ^ 16, n ^ 32 and n ^ 48.
__device__ __forceinline__ int sum_halves(int x) {
  const auto p = __builtin_amdgcn_permlane16_swap((uint32_t)x, (uint32_t)x, false, false);
  const uint32_t s = p[0] + p[1];
  const auto q = __builtin_amdgcn_permlane32_swap(s, s, false, false);
  return (int)(q[0] + q[1]);
}
__device__ __forceinline__ void pieces(float x, _Float16 &hi, _Float16 &lo) {
  hi = (_Float16)x;
  lo = (_Float16)(x - (float)hi);
}
// The same of two values side by side: a packed conversion, two mixed multiply-adds (x
// less a half of the first, which the compiler would form in two steps each) and a
// packed conversion.
__device__ __forceinline__ void pieces2(float x, float y, uint32_t &hi, uint32_t &lo) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  hi = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){x, y}, h2));
  float rx, ry;
  asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(rx) : "v"(hi), "v"(x));
  asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(ry) : "v"(hi), "v"(y));
  lo = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){rx, ry}, h2));
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
// A tile of T rows: its sequence, its first row among the sequence's, the
// sequence's rows, first row of q, tokens and cached tokens; the units of keys in
// each of the sequence's ranges, and the place of the tile's first range among all
// (tile, range) items, and from each range to its next: a sequence's items are its tiles' first ranges, then
// their second ones, and so on, so that neighbours are about as long (workgroups are handed to one group of CUs
// after the other in order, and wait where that one is full: if every second one is short, half of
// the CUs stand idle.  8 prompts of 250 tokens 63.5 -> 56.0 us).
struct Rows { int b, r0, rows, first, n, len, per, item0, stride; };

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }
// The ranges of `per` units that `keys` keys make.
__device__ __forceinline__ int ranges_of(int keys, int unit, int per) {
  return max(1, ceil_div(ceil_div(keys, unit), per));
}
// Sums over lanes 0 .. n of the wave, by DPP: shifts within rows of 16, then the last
// lane of each row to the rows behind it (a shuffle through LDS takes some 100
// cycles, and a search has a dozen of them one after another).
template <int CTRL, int ROWS, typename T>
__device__ __forceinline__ T shifted(T x) {
  return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, ROWS, 0xF, false));
}
template <typename T>
__device__ __forceinline__ T sums_to(T x) {
  x += shifted<0x111, 0xF>(x);
  x += shifted<0x112, 0xF>(x);
  x += shifted<0x114, 0xF>(x);
  x += shifted<0x118, 0xF>(x);
  x += shifted<0x142, 0xA>(x);
  x += shifted<0x143, 0xC>(x);
  return x;
}
__device__ __forceinline__ int of_lane(int x, int l) { return __builtin_amdgcn_readlane(x, l); }
// Sequence b's first row, tokens and cached tokens; nothing beyond the last.
__device__ __forceinline__ void sequence(const AttnArgs &a, int b, int &first, int &n, int &len) {
  first = b;
  n = len = 0;
  if (b >= a.B) return;
  len = min(max(a.kv_len[b], 0), a.width << a.c.shift);
  n = 1;
  if (a.cu) {
    first = min(max(a.cu[b], 0), a.M);
    n = min(max(a.cu[b + 1], first), a.M) - first;
    if (n * a.G <= a.above || n * a.G > a.upto) n = 0;
  }
}

// The units of a range so that about kItems workgroups share `units` of them for each head
// evenly, however long each sequence is.
__device__ __forceinline__ int units_each(float units, int heads) {
  return max(1, (int)fminf(ceilf(units * (float)heads * (1.f / kItems)), 1e9f));
}
// The ranges of a sequence of `len` keys, and `mine`, the units of each: `per`, or more where they would be
// more than kMaxRanges.
__device__ __forceinline__ int ranges_in(int len, int unit, int per, int &mine) {
  mine = max(per, ceil_div(ceil_div(len, unit), kMaxRanges));
  return ranges_of(len, unit, mine);
}

// Tile or item number `at` as find_rows has it, from the index of many sequences (attn_index_kernel): the units of a range, then for each sequence
// the items, and the tiles, of it and those in front of it.  Each step cuts what is left to a
// 64th, a lane each: four steps for 2^20 sequences.
template <int T, bool ITEMS>
__device__ __forceinline__ bool find_indexed(const AttnArgs &a, int at, int unit, Rows &r, int &split) {
  const int32_t *items_to = a.index + kIndexHead, *tiles_to = items_to + a.B, *upto = ITEMS ? items_to : tiles_to;
  const int lane = threadIdx.x & 63;
  int lo = 0, n = a.B;
  while (n > 0) {
    const int step = (n + 63) >> 6;
    const uint64_t past = __ballot(upto[lo + min((lane + 1) * step, n) - 1] > at);
    if (!past) return false;
    const int l = uniform(__ffsll((unsigned long long)past) - 1), skip = l * step;
    lo += skip;
    if (step == 1) break;
    n = min(step, n - skip);
  }
  sequence(a, lo, r.first, r.n, r.len);
  r.b = lo;
  r.first = uniform(r.first);
  r.n = uniform(r.n);
  r.len = uniform(r.len);
  r.rows = r.n * a.G;
  int mine;
  ranges_in(r.len, unit, a.index[0], mine);
  r.per = uniform(mine);
  const int in = uniform(at - (lo ? upto[lo - 1] : 0));
  r.stride = ceil_div(r.rows, T);
  split = ITEMS ? uniform(in / r.stride) : 0;
  const int tile = in - split * r.stride;
  r.r0 = tile * T;
  r.item0 = uniform((lo ? items_to[lo - 1] : 0) + tile);
  return true;
}

// Tile number `at`, or with ITEMS the item number `at`, whose range goes to
// `split`.  Called by whole waves; false where there is none.  The sequences are
// summed over the wave, 64 at a time: first their units, which give the units of a
// range, then their items.
template <int T, bool ITEMS>
__device__ __forceinline__ bool find_rows(const AttnArgs &a, int at, int unit, Rows &r, int &split) {
  if (a.index) return find_indexed<T, ITEMS>(a, at, unit, r, split);
  const int lane = threadIdx.x & 63;
  int per = 1 << 30;
  int first, n, len;
  if (a.splits > 1) {
    float units = 0.f;  // (some 2^30 times 2^16 at the most)
    for (int b0 = 0; b0 < a.B; b0 += 64) {
      sequence(a, b0 + lane, first, n, len);
      units += (float)ceil_div(n * a.G, T) * (float)ceil_div(len, unit);
    }
    units = sums_to(units);  // (lane 63 has them all)
    per = of_lane(units_each(units, a.c.heads), 63);
  }
  int left = at, items0 = 0;
  for (int b0 = 0;; b0 += 64) {
    if (b0 >= a.B) return false;
    if (a.B > 64 || a.splits == 1) sequence(a, b0 + lane, first, n, len);  // (else held from above)
    int mine;
    const int tiles = ceil_div(n * a.G, T), ranges = ranges_in(len, unit, per, mine), items = tiles * ranges;
    const int items_to = sums_to(items), tiles_to = ITEMS ? 0 : sums_to(tiles);
    const int upto = ITEMS ? items_to : tiles_to;
    const uint64_t past = __ballot(upto > left);
    if (past) {
      const int l = uniform(__ffsll((unsigned long long)past) - 1);
      const int in = left - of_lane(upto - (ITEMS ? items : tiles), l);
      r.stride = of_lane(tiles, l);
      split = ITEMS ? uniform(in / r.stride) : 0;
      const int tile = in - split * r.stride;
      r.b = b0 + l;
      r.r0 = tile * T;
      r.first = of_lane(first, l);
      r.n = of_lane(n, l);
      r.len = of_lane(len, l);
      r.per = of_lane(mine, l);
      r.rows = r.n * a.G;
      r.item0 = items0 + of_lane(items_to - items, l) + tile;
      return true;
    }
    left -= of_lane(upto, 63);
    items0 += of_lane(items_to, 63);
  }
}
// Tile `tile` where every sequence has one row and there are too many of them to
// search: found by number, ranges by the sequence's own length.
template <int T>
__device__ __forceinline__ void single_rows(const AttnArgs &a, int tile, int unit, Rows &r) {
  const int per = (a.G + T - 1) / T;
  r.b = r.first = uniform(tile / per);
  r.r0 = (tile - r.b * per) * T;
  r.n = 1;
  r.rows = a.G;
  int first, n, len;
  sequence(a, r.b, first, n, len);
  r.len = uniform(len);
  r.per = uniform(max(kLongRange, ceil_div(ceil_div(r.len, unit), a.splits)));
  r.item0 = tile;
  r.stride = a.tiles;
}

// ---- keys
// The units [u0, u1) of range `split` of a tile that sees `keys` keys, and the
// ranges it has.
struct Range { int u0, u1, ranges; };
__device__ __forceinline__ Range range_at(int keys, int unit, int per, int split) {
  const int units = (keys + unit - 1) / unit;
  // (a division runs in vector registers)
  Range r;
  r.ranges = uniform(ranges_of(keys, unit, per));
  r.u0 = min(units, split * per);
  r.u1 = min(units, r.u0 + per);
  return r;
}

}  // namespace aq
