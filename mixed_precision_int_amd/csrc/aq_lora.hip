// Low-rank adapters of many requests at once beside a shared projection:
//   Y[m,n] = Yin[m,n] + scale[a] sum_{r < rank[a]} B[a][n,r] sum_k A[a][r,k] X[m,k],
// a = ids[m]; a token whose id is outside 0 .. L-1 has no adapter.
//
// Two launches: `shrink` forms v = A x (KS partial sums over column ranges),
// `expand` adds scale B v to the projection's output.  Both run on
// v_mfma_f32_16x16x4_f32 (products and sums in FP32; the adapters' BF16 or
// FP16 values are exact there) over 16 tokens at a time; where these
// belong to several adapters, the adapters are passed over one after
// another and each token keeps the pass that is its own.  A token is one
// column of the products, so neither the order of the tokens nor the mix of
// adapters, nor another request's values, changes its result.
//
// Bound: memory.  X and Yin are read and Y is written once; a rank-16
// adapter does 8 multiply-adds per byte of them.

#include <hip/hip_fp16.h>

#include "aq_device.h"
#include "aq_routed.h"

namespace aq {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

struct bf16_t { uint16_t bits; };

// 8 consecutive adapter values as FP32.
__device__ __forceinline__ void load8f(const float *p, float (&o)[8]) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
  o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
}
__device__ __forceinline__ void load8f(const bf16_t *p, float (&o)[8]) {
  const uint4 v = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = __uint_as_float(w[i] << 16);
    o[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8f(const __half *p, float (&o)[8]) {
  const uint4 v = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = *reinterpret_cast<const __half2 *>(&w[i]);
    o[2 * i] = __low2float(h);
    o[2 * i + 1] = __high2float(h);
  }
}
__device__ __forceinline__ void load4f(const float *p, float (&o)[4]) {
  const float4 a = *reinterpret_cast<const float4 *>(p);
  o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
}
__device__ __forceinline__ void load4f(const bf16_t *p, float (&o)[4]) {
  const uint2 v = *reinterpret_cast<const uint2 *>(p);
  o[0] = __uint_as_float(v.x << 16);
  o[1] = __uint_as_float(v.x & 0xFFFF0000u);
  o[2] = __uint_as_float(v.y << 16);
  o[3] = __uint_as_float(v.y & 0xFFFF0000u);
}
__device__ __forceinline__ void load4f(const __half *p, float (&o)[4]) {
  const uint2 v = *reinterpret_cast<const uint2 *>(p);
  const __half2 a = *reinterpret_cast<const __half2 *>(&v.x), b = *reinterpret_cast<const __half2 *>(&v.y);
  o[0] = __low2float(a); o[1] = __high2float(a);
  o[2] = __low2float(b); o[3] = __high2float(b);
}

// The adapter of token m0 + i16 (-1: none) for every lane.
__device__ __forceinline__ int token_adapter(const LoraArgs &a, int m0, int i16) {
  const int m = m0 + i16;
  const int id = m < a.M ? a.ids[m] : -1;
  return (unsigned)id < (unsigned)a.L ? id : -1;
}

// shrink: one workgroup of 4 waves per 16 tokens x column range; the waves
// take a quarter of the range each, their sums meet in LDS in order.
// RT: 16-rank tiles.
template <typename T, int RT>
__global__ __launch_bounds__(256) void lora_shrink_kernel(const LoraArgs a) {
  __shared__ float4 red[4][RT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  const int m0 = blockIdx.x * 16;
  const int id = token_adapter(a, m0, i16);
  uint32_t rem = (uint32_t)__ballot(id >= 0) & 0xFFFFu;
  if (rem == 0u) return;  // expand does not read these tokens' sums
  const int nb = a.K >> 6;
  const int parts = a.KS * 4, part = blockIdx.y * 4 + wave;
  const int b0 = (int)((long long)nb * part / parts), b1 = (int)((long long)nb * (part + 1) / parts);
  const float *x = a.X + (size_t)min(m0 + i16, a.M - 1) * a.K;
  v4f own[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) own[r] = v4f{0.f, 0.f, 0.f, 0.f};
  while (rem) {
    const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(rem));
    const bool mine = id == ad;
    rem &= ~(uint32_t)__ballot(mine);
    const int rank = a.rank ? min(max(a.rank[ad], 0), a.R) : a.R;
    v4f acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = v4f{0.f, 0.f, 0.f, 0.f};
    const T *A = static_cast<const T *>(a.A) + (size_t)ad * a.R * a.K;
    for (int b = b0; b < b1; ++b) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int k = b * 64 + 32 * q + 8 * g;
        float xv[8];
        if (mine) load8f(x + k, xv);
        else
#pragma unroll
          for (int t = 0; t < 8; ++t) xv[t] = 0.f;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          float wv[8];
          const int row = r * 16 + i16;
          if (row < rank) load8f(A + (size_t)row * a.K + k, wv);
          else
#pragma unroll
            for (int t = 0; t < 8; ++t) wv[t] = 0.f;
#pragma unroll
          for (int t = 0; t < 8; ++t) acc[r] = __builtin_amdgcn_mfma_f32_16x16x4f32(wv[t], xv[t], acc[r], 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < 4; ++t) own[r][t] = mine ? acc[r][t] : own[r][t];
  }
  // lane: ranks 16r + 4g .. + 3 of token i16
#pragma unroll
  for (int r = 0; r < RT; ++r) red[wave][r][lane] = make_float4(own[r][0], own[r][1], own[r][2], own[r][3]);
  __syncthreads();
  for (int r = wave; r < RT; r += 4) {
    float4 s = red[0][r][lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      const float4 p = red[w][r][lane];
      s.x += p.x; s.y += p.y; s.z += p.z; s.w += p.w;
    }
    const int k = 16 * r + 4 * g;
    if (m0 + i16 < a.M && k < a.R)
      *reinterpret_cast<float4 *>(a.v + ((size_t)blockIdx.y * a.M + m0 + i16) * a.R + k) = s;
  }
}

// expand: one wave per 16 tokens x 64 output features (4 waves side by side).
template <typename T, int RT>
__global__ __launch_bounds__(256) void lora_expand_kernel(const LoraArgs a) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  const int m0 = blockIdx.x * 16;
  const int nbk = a.N >> 6;
  const int id = token_adapter(a, m0, i16);
  const uint32_t any = (uint32_t)__ballot(id >= 0) & 0xFFFFu;
  if (any == 0u && a.Yin == a.Y) return;
  // the lane's part of v: ranks 16r + 4g .. + 3 of token i16, times scale
  float v[RT][4];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    v[r][0] = v[r][1] = v[r][2] = v[r][3] = 0.f;
    const int k = 16 * r + 4 * g;
    if (id >= 0 && k < a.R) {
      for (int s = 0; s < a.KS; ++s) {
        const float4 p = *reinterpret_cast<const float4 *>(a.v + ((size_t)s * a.M + m0 + i16) * a.R + k);
        v[r][0] += p.x; v[r][1] += p.y; v[r][2] += p.z; v[r][3] += p.w;
      }
      const float sc = a.scale ? a.scale[id] : 1.f;
#pragma unroll
      for (int t = 0; t < 4; ++t) v[r][t] *= sc;
    }
  }
  const bool stored = m0 + i16 < a.M;
  for (int nb = blockIdx.y * 4 + wave; nb < nbk; nb += gridDim.y * 4) {
    const size_t row = min(m0 + i16, a.M - 1), col = nb * 64 + 4 * g;
    const float *yi = a.Yin + row * a.ldyin + col;
    float *yo = a.Y + row * a.ldy + col;
    v4f own[4];
    float4 y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      own[j] = v4f{0.f, 0.f, 0.f, 0.f};
      y[j] = *reinterpret_cast<const float4 *>(yi + 16 * j);
    }
    uint32_t rem = any;
    while (rem) {
      const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(rem));
      const bool mine = id == ad;
      rem &= ~(uint32_t)__ballot(mine);
      const int rank = a.rank ? min(max(a.rank[ad], 0), a.R) : a.R;
      const T *B = static_cast<const T *>(a.B) + ((size_t)ad * a.N + nb * 64) * a.R;
      v4f acc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int k = 16 * r + 4 * g;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float w[4] = {0.f, 0.f, 0.f, 0.f};
          if (k < rank) {
            load4f(B + (size_t)(16 * j + i16) * a.R + k, w);
#pragma unroll
            for (int t = 1; t < 4; ++t)
              if (k + t >= rank) w[t] = 0.f;
          }
#pragma unroll
          for (int t = 0; t < 4; ++t)
            acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(w[t], v[r][t], acc[j], 0, 0, 0);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int t = 0; t < 4; ++t) own[j][t] = mine ? acc[j][t] : own[j][t];
    }
    // lane: features nb*64 + 16j + 4g .. + 3 of token i16
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (stored)
        *reinterpret_cast<float4 *>(yo + 16 * j) =
            make_float4(y[j].x + own[j][0], y[j].y + own[j][1], y[j].z + own[j][2], y[j].w + own[j][3]);
  }
}

template <typename T, int RT>
hipError_t launch_rt(const LoraArgs &a, hipStream_t stream) {
  const int mt = (a.M + 15) / 16;
  hipLaunchKernelGGL((lora_shrink_kernel<T, RT>), dim3(mt, a.KS), dim3(256), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int nq = (a.N / 64 + 3) / 4;
  hipLaunchKernelGGL((lora_expand_kernel<T, RT>), dim3(mt, nq), dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const LoraArgs &a, hipStream_t stream) {
  if (a.R <= 16) return launch_rt<T, 1>(a, stream);
  if (a.R <= 32) return launch_rt<T, 2>(a, stream);
  if (a.R <= 64) return launch_rt<T, 4>(a, stream);
  return launch_rt<T, 8>(a, stream);
}

}  // namespace

hipError_t launch_lora(const LoraArgs &a, hipStream_t stream) {
  switch (a.type) {
    case AQ_TYPE_F32: return launch_t<float>(a, stream);
    case AQ_TYPE_BF16: return launch_t<bf16_t>(a, stream);
    default: return launch_t<__half>(a, stream);
  }
}

}  // namespace aq
