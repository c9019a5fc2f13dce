// Norm and gate into INT8 rows (aq_norm_quant, aq_swiglu_quant).
//
// One workgroup per row, the row in registers: read once, written once as
// codes.  Both end in aq_quant_act's rule (aq_quant.h), so the FP32 value in
// front of it has to be the definition's to the last bit, or a code next to a
// tie turns over: the arithmetic is FP64, rounded once.
//
// Many rows are bound by memory: the norm of 8192 x 5120 FP32 rows with their residual, 545 MB,
// takes 103 us (5.3 TB/s), the gate of 2048 x 9728, 179 MB, 39 us (4.6; a copy of 4 GiB moves 4.4 to
// 4.8 TB/s).  Few are bound by their row's chain, load, sum, maximum, codes (one row of 4096: 4.0 us),
// the gate's by the FP64 exponential and division on one CU (5 rows of 14336: 8.2 us).

#include <type_traits>

#include "aq_layer.h"
#include "aq_quant.h"

namespace aq {
namespace {

typedef unsigned short us4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t f32_to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
__device__ __forceinline__ float f16_to_f32(uint16_t b) {
  return (float)__builtin_bit_cast(_Float16, b);
}
__device__ __forceinline__ uint16_t f32_to_f16(float f) {
  return __builtin_bit_cast(uint16_t, (_Float16)f);
}

// Four values at 4 * c of a row of type TYPE.
template <int TYPE>
__device__ __forceinline__ float4 load4(const void *row, int c) {
  if constexpr (TYPE == AQ_TYPE_F32) {
    return static_cast<const float4 *>(row)[c];
  } else {
    const us4 b = static_cast<const us4 *>(row)[c];
    if constexpr (TYPE == AQ_TYPE_BF16)
      return make_float4(bf16_to_f32(b.x), bf16_to_f32(b.y), bf16_to_f32(b.z), bf16_to_f32(b.w));
    else
      return make_float4(f16_to_f32(b.x), f16_to_f32(b.y), f16_to_f32(b.z), f16_to_f32(b.w));
  }
}

// h rounded to TYPE.
template <int TYPE>
__device__ __forceinline__ float round_to(float h) {
  if constexpr (TYPE == AQ_TYPE_BF16) return bf16_to_f32(f32_to_bf16(h));
  if constexpr (TYPE == AQ_TYPE_F16) return f16_to_f32(f32_to_f16(h));
  return h;
}
template <int TYPE>
__device__ __forceinline__ void store4(void *row, int c, const float4 &h) {
  if constexpr (TYPE == AQ_TYPE_F32) {
    static_cast<float4 *>(row)[c] = h;
  } else if constexpr (TYPE == AQ_TYPE_BF16) {
    const us4 b = {f32_to_bf16(h.x), f32_to_bf16(h.y), f32_to_bf16(h.z), f32_to_bf16(h.w)};
    static_cast<us4 *>(row)[c] = b;
  } else {
    const us4 b = {f32_to_f16(h.x), f32_to_f16(h.y), f32_to_f16(h.z), f32_to_f16(h.w)};
    static_cast<us4 *>(row)[c] = b;
  }
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
// Sum over the workgroup, the waves' sums added in order.
template <int T>
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[T / 64];
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double r = red[0];
#pragma unroll
  for (int w = 1; w < T / 64; ++w) r += red[w];
  return r;
}

// Codes and scale of the row whose values v (float4 i at column threadIdx.x +
// i * T) the workgroup holds.
template <int T, int NV>
__device__ __forceinline__ void quant_row(const float4 (&v)[NV], uint32_t amax, int n4, float *Y, int8_t *qx,
                                          float *sx) {
  const uint32_t top = block_max_u32<T>(amax);
  // (the rule's maximum with 1e-12 would hide a NaN)
  const double s = top < 0x7F800000u ? row_scale(top) : (double)__uint_as_float(top);
  if (threadIdx.x == 0) *sx = (float)s;
  const float inv = (float)(1.0 / s);
  uint32_t *out = reinterpret_cast<uint32_t *>(qx);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * T;
    if (c < n4) {
      out[c] = codes4_fast(v[i], s, inv);
      if (Y) reinterpret_cast<float4 *>(Y)[c] = v[i];
    }
  }
}

template <int TYPE, int T, int NV>
__global__ __launch_bounds__(T) void norm_quant_kernel(NormArgs a) {
  const size_t at = (size_t)blockIdx.x * a.H;
  const size_t bytes = TYPE == AQ_TYPE_F32 ? 4 : 2;
  const int n4 = a.H >> 2;
  const char *x = static_cast<const char *>(a.X) + at * bytes;
  const char *r = a.R ? static_cast<const char *>(a.R) + at * bytes : nullptr;
  char *h = a.Hout ? static_cast<char *>(a.Hout) + at * bytes : nullptr;
  float4 v[NV];
  double sum = 0.;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * T;
    v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < n4) {
      v[i] = load4<TYPE>(x, c);
      if (r) {
        const float4 b = load4<TYPE>(r, c);
        v[i] = make_float4(round_to<TYPE>(v[i].x + b.x), round_to<TYPE>(v[i].y + b.y),
                           round_to<TYPE>(v[i].z + b.z), round_to<TYPE>(v[i].w + b.w));
      }
      if (h) store4<TYPE>(h, c, v[i]);
    }
    sum += (double)v[i].x * v[i].x + (double)v[i].y * v[i].y + (double)v[i].z * v[i].z + (double)v[i].w * v[i].w;
  }
  const double n = 1. / sqrt(block_sum<T>(sum) / a.H + a.eps);
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * T;
    if (c < n4) {
      const float4 w = a.w_type == AQ_TYPE_F32    ? load4<AQ_TYPE_F32>(a.W, c)
                       : a.w_type == AQ_TYPE_BF16 ? load4<AQ_TYPE_BF16>(a.W, c)
                                                  : load4<AQ_TYPE_F16>(a.W, c);
      v[i] = make_float4((float)(v[i].x * n * w.x), (float)(v[i].y * n * w.y), (float)(v[i].z * n * w.z),
                         (float)(v[i].w * n * w.w));
    }
    amax = max(amax, abs_bits4(v[i]));
  }
  quant_row<T, NV>(v, amax, n4, a.Y ? a.Y + at : nullptr, a.qx + at, a.sx + blockIdx.x);
}

__device__ __forceinline__ float gate(float g, float u) { return (float)(g / (1. + exp(-(double)g)) * u); }

template <int T, int NV>
__global__ __launch_bounds__(T) void swiglu_quant_kernel(SwigluArgs a) {
  const int n4 = a.I >> 2;
  const float4 *g = reinterpret_cast<const float4 *>(a.GU + (size_t)blockIdx.x * a.ld);
  const float4 *u = g + n4;
  float4 v[NV];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = threadIdx.x + i * T;
    v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < n4) {
      const float4 p = g[c], q = u[c];
      v[i] = make_float4(gate(p.x, q.x), gate(p.y, q.y), gate(p.z, q.z), gate(p.w, q.w));
    }
    amax = max(amax, abs_bits4(v[i]));
  }
  const size_t at = (size_t)blockIdx.x * a.I;
  quant_row<T, NV>(v, amax, n4, a.Y ? a.Y + at : nullptr, a.qx + at, a.sx + blockIdx.x);
}

// Float4 groups per thread: every thread holds NV of them, so that a row's length rounds
// up to one of these.
template <int NV>
using Groups = std::integral_constant<int, NV>;
template <int T, typename F>
hipError_t with_groups(int nv, F f) {
  if constexpr (T != 512) {
    if (nv <= 1) return f(Groups<1>());
    if (nv <= 2) return f(Groups<2>());
  }
  if (nv <= 3) return f(Groups<3>());
  if (nv <= 4) return f(Groups<4>());
  if constexpr (T != 256) {
    if (nv <= 5) return f(Groups<5>());
    if (nv <= 6) return f(Groups<6>());
    if (nv <= 8) return f(Groups<8>());
  }
  return hipErrorInvalidValue;
}
// Threads of a row: with few rows as many as there may be, since a row's arithmetic is one CU's (the gate of one
// row of 9728: 8.5 us with 256 threads, 6.3 with 1024); with many, so few that several rows share a CU and so
// many that a thread's values leave room for them.  Norm of 8192 rows, us with 256 | 512 | 1024
// threads: of 2560 43 | 48 | 64, of 4096 78 | 76 | 91, of 5120 100 | 94 | 111, of 16384 407 | 318 | 339; gate: of 4096
// 70 | 72 | 78, of 9728 156 | 153 | 162, of 14336 231 | 220 | 232.  256 rows of 4096: 6.1 | 5.4 | 5.7, of 16384
// 18 | 14 | 13; 512 rows of 4096: 7.8 | 7.2 | 8.5.
template <typename F>
hipError_t with_threads(int M, int n, F f) {
  if (M < 256 || n > 16384) return f(std::integral_constant<int, 1024>());
  return n > 4096 ? f(std::integral_constant<int, 512>()) : f(std::integral_constant<int, 256>());
}

}  // namespace

hipError_t launch_norm_quant(const NormArgs &a, hipStream_t stream) {
  return with_threads(a.M, a.H, [&](auto threads) {
    constexpr int T = decltype(threads)::value;
    return with_groups<T>((a.H / 4 + T - 1) / T, [&](auto nv) {
      constexpr int NV = decltype(nv)::value;
      const dim3 g(a.M), b(T);
      if (a.type == AQ_TYPE_F32) hipLaunchKernelGGL((norm_quant_kernel<AQ_TYPE_F32, T, NV>), g, b, 0, stream, a);
      else if (a.type == AQ_TYPE_BF16) hipLaunchKernelGGL((norm_quant_kernel<AQ_TYPE_BF16, T, NV>), g, b, 0, stream, a);
      else hipLaunchKernelGGL((norm_quant_kernel<AQ_TYPE_F16, T, NV>), g, b, 0, stream, a);
      return hipGetLastError();
    });
  });
}
hipError_t launch_swiglu_quant(const SwigluArgs &a, hipStream_t stream) {
  return with_threads(a.M, a.I, [&](auto threads) {
    constexpr int T = decltype(threads)::value;
    return with_groups<T>((a.I / 4 + T - 1) / T, [&](auto nv) {
      hipLaunchKernelGGL((swiglu_quant_kernel<T, decltype(nv)::value>), dim3(a.M), dim3(T), 0, stream, a);
      return hipGetLastError();
    });
  });
}

}  // namespace aq
