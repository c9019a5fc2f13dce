// The router's choice of experts by one wave: device code shared by the
// choice kernel and the first kernel of the experts' layer.
#pragma once

#include "aq_device.h"
#include "aq_quant.h"
#include "aq_routed.h"

namespace aq {

// 64-bit integers in the order of the doubles (-inf lowest of the ordered
// values; 0 is below every key and marks a chosen or absent one).
__device__ __forceinline__ uint64_t order_of(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, false);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
__device__ __forceinline__ double readlane_f64(double v, int src) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, src);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), src);
  return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
}
// Sum / maximum over the 64 lanes, returned uniform: DPP within rows of 16
// lanes (quad xor 1, quad xor 2, half-row mirror, row mirror), then the four
// rows by readlane (the wave-wide shuffles of 64-bit values, two LDS
// permutes a step, took several times as long).
__device__ __forceinline__ double wave_sum_f64(double v) {
  v += dpp_f64<0xB1>(v);
  v += dpp_f64<0x4E>(v);
  v += dpp_f64<0x141>(v);
  v += dpp_f64<0x140>(v);
  return (readlane_f64(v, 0) + readlane_f64(v, 16)) + (readlane_f64(v, 32) + readlane_f64(v, 48));
}
__device__ __forceinline__ double wave_max_f64(double v) {
  v = fmax(v, dpp_f64<0xB1>(v));
  v = fmax(v, dpp_f64<0x4E>(v));
  v = fmax(v, dpp_f64<0x141>(v));
  v = fmax(v, dpp_f64<0x140>(v));
  return fmax(fmax(readlane_f64(v, 0), readlane_f64(v, 16)), fmax(readlane_f64(v, 32), readlane_f64(v, 48)));
}

// Maximum over the wave of unsigned values, uniform: DPP within rows of 16
// lanes, then the four rows by readlane.
__device__ __forceinline__ uint32_t wave_max_rows_u32(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
  return max(max((uint32_t)__builtin_amdgcn_readlane((int)v, 0), (uint32_t)__builtin_amdgcn_readlane((int)v, 16)),
             max((uint32_t)__builtin_amdgcn_readlane((int)v, 32), (uint32_t)__builtin_amdgcn_readlane((int)v, 48)));
}

// One wave's choice for one token from its logits l[E] (global or LDS); lane i
// holds experts i, i + 64, ...  Lane j < top_k returns the j-th chosen expert
// (-1: none left) and, if WEIGHTS are asked for, its weight.  Every round takes
// the largest key by the upper 32 bits of its order; where several lanes hold
// these, by the lower 32 bits among them, then by the lowest expert.
template <int NE>
__device__ __forceinline__ void choose(const RouteArgs &a, const double *l, int lane, bool weights, int &id,
                                       float &weight) {
  double v[NE];
  uint32_t hi[NE], lo[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = lane + 64 * i;
    v[i] = e < a.E ? l[e] : -INFINITY;
  }
  const bool softmax = a.score == AQ_SCORE_SOFTMAX;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = lane + 64 * i;
    const float b = (a.bias && e < a.E) ? a.bias[e] : 0.f;
    if (!softmax) v[i] = 1. / (1. + exp(-v[i]));
    // excluded whatever the logit is (NaN or +inf would come out on top); else
    // NaN above every key, whatever its sign bit
    const double k = v[i] + (double)b;
    const uint64_t key = e >= a.E || b == -INFINITY ? 0 : k != k ? ~0ull : order_of(k);
    hi[i] = (uint32_t)(key >> 32);
    lo[i] = (uint32_t)key;
  }
  const uint64_t none = order_of(-INFINITY);
  id = -1;
  double mine = -INFINITY;  // the chosen logit (softmax) or p (sigmoid)
  for (int j = 0; j < a.top_k; ++j) {
    uint32_t h = hi[0];
#pragma unroll
    for (int i = 1; i < NE; ++i) h = max(h, hi[i]);
    h = wave_max_rows_u32(h);
    // (upper words of -inf and below: nothing but excluded and chosen experts)
    if (h <= (uint32_t)(none >> 32)) break;
    uint64_t has[NE];
    int n = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      has[i] = __ballot(hi[i] == h);
      n += __popcll(has[i]);
    }
    if (n > 1) {  // uniform
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < NE; ++i) m = hi[i] == h ? max(m, lo[i]) : m;
      m = wave_max_rows_u32(m);
#pragma unroll
      for (int i = 0; i < NE; ++i) has[i] = __ballot(hi[i] == h && lo[i] == m);
    }
    int e = -1;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (e < 0 && has[i]) {
        const int src = __builtin_ctzll(has[i]);
        e = 64 * i + src;
        const double p = readlane_f64(v[i], src);
        if (lane == j) mine = p;
        if (lane == src) hi[i] = lo[i] = 0;
      }
    if (lane == j) id = e;
  }
  weight = 0.f;
  if (!weights) return;
  double total = 1.;
  if (softmax) {
    // with norm relative to the largest chosen logit: the chosen experts' ratios
    // survive where their shares of the whole softmax underflow
    double top = mine;
    if (!a.norm) {
#pragma unroll
      for (int i = 0; i < NE; ++i) top = fmax(top, v[i]);
    }
    top = wave_max_f64(top);
    mine = id >= 0 ? exp(mine - top) : 0.;
    if (a.norm) {
      total = wave_sum_f64(mine);
    } else {
      double sum = 0.;
#pragma unroll
      for (int i = 0; i < NE; ++i) sum += exp(v[i] - top);
      total = wave_sum_f64(sum);
    }
  } else {
    if (id < 0) mine = 0.;
    if (a.norm) total = wave_sum_f64(mine);
  }
  // (a total that is NaN is not one of nothing: the token's weights show it)
  weight = id >= 0 && !(total <= 0.) ? (float)((double)a.scale * (mine / total)) : 0.f;
}

}  // namespace aq
