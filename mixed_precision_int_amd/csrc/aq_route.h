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

// One wave's choice for one token from its logits l[E] (global or LDS); lane i
// holds experts i, i + 64, ...  Lane j < top_k returns the j-th chosen expert (-1: none
// left) and its weight.  Every round takes the largest key: the wave maximum
// of its upper 32 bits, of the lower 32 bits among the lanes that hold it
// where these are several, then the lowest expert that holds both.
template <int NE>
__device__ __forceinline__ void choose(const RouteArgs &a, const double *l, int lane, int &id,
                                       float &weight) {
  double v[NE];
  uint64_t key[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = lane + 64 * i;
    v[i] = e < a.E ? l[e] : -INFINITY;
  }
  const bool softmax = a.score == AQ_SCORE_SOFTMAX;
  double top = 0., sum = 0.;
  if (softmax && !a.norm) {
    top = v[0];
#pragma unroll
    for (int i = 1; i < NE; ++i) top = fmax(top, v[i]);
    top = wave_max_f64(top);
#pragma unroll
    for (int i = 0; i < NE; ++i) sum += exp(v[i] - top);
    sum = wave_sum_f64(sum);
  }
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = lane + 64 * i;
    const double b = (a.bias && e < a.E) ? (double)a.bias[e] : 0.;
    if (!softmax) v[i] = 1. / (1. + exp(-v[i]));
    key[i] = e < a.E ? order_of(v[i] + b) : 0;
  }
  const uint64_t none = order_of(-INFINITY);
  id = -1;
  double mine = -INFINITY;  // the chosen logit (softmax) or p (sigmoid)
  for (int j = 0; j < a.top_k; ++j) {
    uint64_t best = key[0];
#pragma unroll
    for (int i = 1; i < NE; ++i) best = key[i] > best ? key[i] : best;
    const uint32_t hi = wave_max_u32((uint32_t)(best >> 32));
    const uint64_t with = __ballot((uint32_t)(best >> 32) == hi);
    const uint32_t lo = (with & (with - 1))
                            ? wave_max_u32((uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u)
                            : (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)best, __builtin_ctzll(with));
    best = ((uint64_t)hi << 32) | lo;
    if (best <= none) break;  // only experts excluded by a bias of -inf are left
    int e = -1;
    double p = 0.;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const uint64_t has = __ballot(key[i] == best);
      if (e < 0 && has) {
        const int src = __builtin_ctzll(has);
        e = 64 * i + src;
        p = readlane_f64(v[i], src);
        if (lane == src) key[i] = 0;
      }
    }
    if (lane == j) {
      id = e;
      mine = p;
    }
  }
  double total = 1.;
  if (softmax) {
    // with norm relative to the largest chosen logit: the chosen experts' ratios
    // survive where their shares of the whole softmax underflow
    if (a.norm) top = wave_max_f64(mine);
    mine = id >= 0 ? exp(mine - top) : 0.;
    total = a.norm ? wave_sum_f64(mine) : sum;
  } else {
    if (id < 0) mine = 0.;
    if (a.norm) total = wave_sum_f64(mine);
  }
  weight = id >= 0 && total > 0. ? (float)((double)a.scale * (mine / total)) : 0.f;
}

}  // namespace aq
