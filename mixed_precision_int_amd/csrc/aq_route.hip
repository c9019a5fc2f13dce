// The router of a mixture-of-experts layer: scores of every token for every
// expert, the top_k of them, and their weights.
//
//   l[m,e] = sum_k X[m,k] Wr[e,k]            (64-bit products and sums)
//   softmax: key = l + b,  p = exp(l - max) / sum exp(l - max)
//   sigmoid: key = p + b,  p = 1 / (1 + exp(-l))
//   ids = the top_k largest keys, equal keys in increasing expert order;
//   w = scale * p[id], with `norm` divided by the sum of the chosen p.
//
// The choice of experts is a comparison of sums, so the sums are formed in
// FP64: an FP32 sum moves a logit by about 1e-6 of its spread and would
// change the choice of one token in some ten thousand against the
// definition.
//
// logits: one workgroup of 8 waves per 16 tokens x 16 experts on
// v_mfma_f64_16x16x4_f64, the input columns cut into 8 contiguous ranges of
// 64-column blocks (one per wave), whose sums are added through LDS in
// increasing order.  Lane l of a wave holds row l % 16 of both operands;
// its 16-byte load at k = 64b + 16q + 4(l / 16) feeds four products, product
// t taking element t of every lane.
// choice: one wave per token.

#include "aq_device.h"
#include "aq_routed.h"

namespace aq {
namespace {

typedef double v4d __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void load4(const float *p, double (&o)[4]) {
  const float4 v = *reinterpret_cast<const float4 *>(p);
  o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
}
__device__ __forceinline__ void load4(const uint16_t *p, double (&o)[4]) {  // bfloat16 bits
  const uint2 v = *reinterpret_cast<const uint2 *>(p);
  o[0] = __uint_as_float(v.x << 16);
  o[1] = __uint_as_float(v.x & 0xFFFF0000u);
  o[2] = __uint_as_float(v.y << 16);
  o[3] = __uint_as_float(v.y & 0xFFFF0000u);
}

constexpr int kRouteWaves = 8;

template <typename TW>
__global__ __launch_bounds__(kRouteWaves * 64) void route_logits_kernel(const RouteArgs a) {
  __shared__ double red[kRouteWaves][256];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  const int m0 = blockIdx.x * 16, e0 = blockIdx.y * 16;
  // rows past the end read the last row; their sums are not stored
  const float *x = a.X + (size_t)min(m0 + i16, a.M - 1) * a.K + 4 * g;
  const TW *w = static_cast<const TW *>(a.Wr) + (size_t)min(e0 + i16, a.E - 1) * a.K + 4 * g;
  const int nb = a.K >> 6;
  const int b0 = nb * wave / kRouteWaves, b1 = nb * (wave + 1) / kRouteWaves;
  v4d acc = {0., 0., 0., 0.};
  for (int b = b0; b < b1; ++b) {
    double xv[4][4], wv[4][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      load4(x + (size_t)b * 64 + 16 * q, xv[q]);
      load4(w + (size_t)b * 64 + 16 * q, wv[q]);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int t = 0; t < 4; ++t) acc = __builtin_amdgcn_mfma_f64_16x16x4f64(xv[q][t], wv[q][t], acc, 0, 0, 0);
  }
  // element t of a lane: token g + 4t, expert i16
#pragma unroll
  for (int t = 0; t < 4; ++t) red[wave][(g + 4 * t) * 16 + i16] = acc[t];
  __syncthreads();
  if (threadIdx.x < 256) {
    const int m = m0 + (threadIdx.x >> 4), e = e0 + (threadIdx.x & 15);
    if (m < a.M && e < a.E) {
      double s = 0.;
#pragma unroll
      for (int i = 0; i < kRouteWaves; ++i) s += red[i][threadIdx.x];
      a.logits[(size_t)m * a.E + e] = s;
    }
  }
}

// 64-bit integers in the order of the doubles (-inf lowest of the ordered
// values; 0 is below every key and marks a chosen or absent one).
__device__ __forceinline__ uint64_t order_of(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint64_t p = __shfl_xor((unsigned long long)v, o);
    v = p > v ? p : v;
  }
  return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// One wave's choice for token m from its logits l[E]; lane i holds experts
// i, i + 64, ...  Lane j < top_k returns the j-th chosen expert (-1: none
// left) and its weight.
template <int NE>
__device__ __forceinline__ void choose(const RouteArgs &a, const double *__restrict__ l, int lane, int &id,
                                       float &weight) {
  double v[NE];
  uint64_t key[NE];
  double top = -INFINITY;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = lane + 64 * i;
    v[i] = e < a.E ? l[e] : -INFINITY;
    top = fmax(top, v[i]);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmax(top, __shfl_xor(top, o));
  double sum = 0.;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = lane + 64 * i;
    const double b = (a.bias && e < a.E) ? (double)a.bias[e] : 0.;
    if (a.score == AQ_SCORE_SOFTMAX) {
      key[i] = order_of(v[i] + b);
      sum += exp(v[i] - top);
    } else {
      v[i] = 1. / (1. + exp(-v[i]));
      key[i] = order_of(v[i] + b);
    }
    if (e >= a.E) key[i] = 0;
  }
  const uint64_t none = order_of(-INFINITY);
  id = -1;
  double mine = -INFINITY;  // the chosen logit (softmax) or p (sigmoid)
  for (int j = 0; j < a.top_k; ++j) {
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < NE; ++i) best = key[i] > best ? key[i] : best;
    best = wave_max_u64(best);
    if (best <= none) break;  // only experts excluded by a bias of -inf are left
    // the first expert that holds it: lowest i, then lowest lane
    int e = -1;
    double p = 0.;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const uint64_t has = __ballot(key[i] == best);
      if (e < 0 && has) {
        const int src = __builtin_ctzll(has);
        e = 64 * i + src;
        p = __shfl(v[i], src);
        if (lane == src) key[i] = 0;
      }
    }
    if (lane == j) {
      id = e;
      mine = p;
    }
  }
  double total = 1.;
  if (a.score == AQ_SCORE_SOFTMAX) {
    // with norm relative to the largest chosen logit: the chosen experts' ratios
    // survive where their shares of the whole softmax underflow
    if (a.norm) {
      top = mine;
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) top = fmax(top, __shfl_xor(top, o));
    }
    mine = id >= 0 ? exp(mine - top) : 0.;
    total = wave_sum(a.norm ? mine : sum);
  } else {
    if (id < 0) mine = 0.;
    if (a.norm) total = wave_sum(mine);
  }
  weight = id >= 0 && total > 0. ? (float)((double)a.scale * (mine / total)) : 0.f;
}

template <int NE>
__global__ __launch_bounds__(256) void route_choice_kernel(const RouteArgs a) {
  const int lane = threadIdx.x & 63;
  const int m = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (m >= a.M) return;
  int id;
  float w;
  choose<NE>(a, a.logits + (size_t)m * a.E, lane, id, w);
  if (lane < a.top_k) {
    a.ids[(size_t)m * a.top_k + lane] = id;
    a.weights[(size_t)m * a.top_k + lane] = w;
  }
}

}  // namespace

hipError_t launch_route(const RouteArgs &a, hipStream_t stream) {
  const dim3 grid((a.M + 15) / 16, (a.E + 15) / 16);
  if (a.wr_type == AQ_TYPE_F32)
    hipLaunchKernelGGL(route_logits_kernel<float>, grid, dim3(kRouteWaves * 64), 0, stream, a);
  else
    hipLaunchKernelGGL(route_logits_kernel<uint16_t>, grid, dim3(kRouteWaves * 64), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 g2((a.M + 3) / 4), b2(256);
  if (a.E <= 64) hipLaunchKernelGGL(route_choice_kernel<1>, g2, b2, 0, stream, a);
  else if (a.E <= 128) hipLaunchKernelGGL(route_choice_kernel<2>, g2, b2, 0, stream, a);
  else if (a.E <= 256) hipLaunchKernelGGL(route_choice_kernel<4>, g2, b2, 0, stream, a);
  else hipLaunchKernelGGL(route_choice_kernel<16>, g2, b2, 0, stream, a);
  return hipGetLastError();
}

}  // namespace aq
