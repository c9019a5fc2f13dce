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
// logits, up to 2048 pairs: one wave per expert and token on the vector ALU,
// lane l taking columns 256c + 4l .. + 3 of both rows, so that a row is one
// coalesced stream and a call is about one load round trip; the lanes' FP64
// sums are added across the wave.
// logits, more: 32 x 32 tiles on v_mfma_f64_16x16x4_f64 over column ranges,
// whose partial sums the choice adds in increasing order.  Lane l of a wave
// holds row l % 16 of both operands; its 4 values at k = 16q + 4(l / 16) feed
// four products, product t taking element t of every lane.
// choice: one wave per token.

#include <type_traits>

#include "aq_lds_pipe.h"
#include "aq_route.h"

namespace aq {
namespace {

typedef double v4d __attribute__((ext_vector_type(4)));

// 4 consecutive values, widened.
__device__ __forceinline__ void widen4(const v4f &v, double (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = v[i];
}
__device__ __forceinline__ void widen4(const v2u &v, double (&o)[4]) {  // bfloat16 bits
  o[0] = __uint_as_float(v[0] << 16);
  o[1] = __uint_as_float(v[0] & 0xFFFF0000u);
  o[2] = __uint_as_float(v[1] << 16);
  o[3] = __uint_as_float(v[1] & 0xFFFF0000u);
}
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

// Quantizes token row m with the whole workgroup of T threads: aq_quant_act's
// rule, the row's largest magnitude, then the codes from a second read, which
// finds the row in the first-level cache.
template <int T>
__device__ __forceinline__ void quant_row(const RouteArgs &a, int m, int8_t *__restrict__ qx, float *__restrict__ sx) {
  if (m >= a.M) return;
  const float4 *row = reinterpret_cast<const float4 *>(a.X + (size_t)m * a.K);
  const int n4 = a.K >> 2;
  uint32_t amax = 0;
#pragma unroll 4
  for (int c = threadIdx.x; c < n4; c += T) amax = max(amax, abs_bits4(row[c]));
  const double s = row_scale(block_max_u32<T>(amax));
  if (threadIdx.x == 0) sx[m] = (float)s;
  const float inv = (float)(1.0 / s);
  uint32_t *out = reinterpret_cast<uint32_t *>(qx + (size_t)m * a.K);
#pragma unroll 4
  for (int c = threadIdx.x; c < n4; c += T) out[c] = codes4_fast(row[c], s, inv);
}

// A 1 KB piece of a tile: 64 lanes x 16 bytes from the lanes' addresses to
// consecutive LDS bytes.
__device__ __forceinline__ void piece(__amdgpu_buffer_rsrc_t r, void *lds, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)lds, 16, voff, soff, 0, 0);
}

// One workgroup of 4 waves per 32 tokens x 32 experts and column range; blocks
// past the tiles quantize one token row each (qx != nullptr).
//   Each wave takes 16 of a step's 64 columns for the whole tile, so that an
// operand is widened once per two products and the four accumulators do not
// wait for each other (with a quarter of the tile per wave 38 us, so 35 us, for
// 1024 x 5120 x 160; the products alone are 21 us at the matrix cores' rate);
// the waves' sums meet in LDS at the end.
//   Both operands go through LDS in steps of 64 columns, two steps deep, by
// loads whose lanes read whole 128-byte lines (the MFMA operand read straight
// from memory takes 64 bytes of each of 16 rows a power of two apart, which
// collide in the first-level cache: 58 us, with or without the products).  16-byte granule q of row r sits at place q ^ r, so
// that the 16 rows of an operand read fall in different banks.
template <typename TW>
__global__ __launch_bounds__(256, 4) void route_tile_kernel(const RouteArgs a, int8_t *__restrict__ qx,
                                                         float *__restrict__ sx) {
  constexpr int ST = 2, XB = 32 * 256, WROW = 64 * sizeof(TW), WB = 32 * WROW;
  constexpr int WG = WROW / 16;               // granules of an expert's row step
  __shared__ __align__(16) uint8_t lds[ST][XB + WB];
  const int mt = (a.M + 31) / 32, et = (a.E + 31) / 32;
  int id = blockIdx.x;
  if (id >= mt * et * a.KS) return quant_row<256>(a, id - mt * et * a.KS, qx, sx);
  const int ks = id % a.KS;
  id /= a.KS;
  const int m0 = (id / et) * 32, e0 = (id % et) * 32;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  const int nb = a.K >> 6;
  const int b0 = (int)((long long)nb * ks / a.KS), b1 = (int)((long long)nb * (ks + 1) / a.KS);
  // rows past the end read the last row; their sums are not stored
  const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<float *>(a.X + (size_t)m0 * a.K), 0, 0x7FFFFFFF, 0x00020000);
  const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<TW *>(static_cast<const TW *>(a.Wr) + (size_t)e0 * a.K), 0, 0x7FFFFFFF, 0x00020000);
  int xoff[2], woff[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = (2 * wave + i) * 4 + (lane >> 4);  // X: 4 rows of 16 granules a piece
    xoff[i] = min(r, a.M - 1 - m0) * a.K * 4 + 16 * ((lane & 15) ^ (r & 15));
    const int wr = ((WB / 4096) * wave + i) * (64 / WG) + lane / WG;
    woff[i] = min(wr, a.E - 1 - e0) * a.K * (int)sizeof(TW) + 16 * ((lane % WG) ^ (wr & (WG - 1)));
  }
  auto fetch = [&](int b, int at) __attribute__((always_inline)) {
    b = min(b, b1 - 1);  // past the range: the last step again (never multiplied)
#pragma unroll
    for (int i = 0; i < 2; ++i) piece(rx, lds[at] + (2 * wave + i) * 1024, xoff[i], b * 256);
#pragma unroll
    for (int i = 0; i < WB / 4096; ++i) piece(rw, lds[at] + XB + ((WB / 4096) * wave + i) * 1024, woff[i], b * WROW);
  };
  // the wave's 16 columns of a step, rows i16 and 16 + i16 of both operands:
  // the lane's pieces in stage 0
  typedef std::conditional_t<sizeof(TW) == 4, v4f, v2u> Wv;
  uint32_t xa[2], wa[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    xa[i] = lds_address(lds) + (16 * i + i16) * 256 + 16 * ((4 * wave + g) ^ i16);
    wa[i] = lds_address(lds) + XB + (16 * i + i16) * WROW +
            (sizeof(TW) == 4 ? 16 * ((4 * wave + g) ^ i16) : 16 * ((2 * wave + (g >> 1)) ^ (i16 & 7)) + 8 * (g & 1));
  }
  v4d acc[2][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i >> 1][i & 1] = v4d{0., 0., 0., 0.};
  fetch(b0, 0);
  int at = 0;
  for (int b = b0; b < b1; ++b) {
    // this step's pieces have landed, for every wave, and every wave has read
    // the other place
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0), lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    fetch(b + 1, at ^ 1);
    const uint32_t xs[2] = {xa[0] + at * (XB + WB), xa[1] + at * (XB + WB)};
    const uint32_t ws[2] = {wa[0] + at * (XB + WB), wa[1] + at * (XB + WB)};
    v4f xq[2];
    Wv wq[2];
    lds_read(xs, ws, xq, wq);
    double xv[2][4], wv[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      widen4(xq[i], xv[i]);
      widen4(wq[i], wv[i]);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[i >> 1][i & 1] = __builtin_amdgcn_mfma_f64_16x16x4f64(xv[i >> 1][t], wv[i & 1][t], acc[i >> 1][i & 1], 0, 0, 0);
    at ^= 1;
  }
  // no load into LDS stays open; the waves' sums meet there, wave w finishing
  // tokens 16 (w % 2) .. and experts 16 (w / 2) ..
  __builtin_amdgcn_s_waitcnt(0x0070);
  __syncthreads();
  double *red = reinterpret_cast<double *>(lds);  // [wave][one of the three other waves'][element][lane]
  static_assert(sizeof(lds) >= 4 * 3 * 4 * 64 * sizeof(double), "");
  v4d own = acc[0][0];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i == wave) {
      own = acc[i & 1][i >> 1];
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t) red[((wave * 3 + ((i - wave - 1) & 3)) * 4 + t) * 64 + lane] = acc[i & 1][i >> 1][t];
    }
  }
  __syncthreads();
  // r[d]: the sums of wave + d (mod 4), which holds this tile as its other of place
  // (-d - 1) mod 4
  double r[4][4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    r[0][t] = own[t];
#pragma unroll
    for (int d = 1; d < 4; ++d) r[d][t] = red[((((wave + d) & 3) * 3 + ((3 - d) & 3)) * 4 + t) * 64 + lane];
  }
  // element t of a lane: token g + 4t, expert i16.  Added in the order of the waves
  // (of their columns) everywhere: in that of d it would go by the place in the
  // tile, and equal rows of Wr 16 apart get sums that differ in their last bit.
  const int e = e0 + (wave >> 1) * 16 + i16;
  auto store = [&](const double (&p0)[4], const double (&p1)[4], const double (&p2)[4],
                   const double (&p3)[4]) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int m = m0 + (wave & 1) * 16 + g + 4 * t;
      if (m < a.M && e < a.E) a.logits[((size_t)ks * a.M + m) * a.E + e] = ((p0[t] + p1[t]) + p2[t]) + p3[t];
    }
  };
  switch (wave) {
    case 0: return store(r[0], r[1], r[2], r[3]);
    case 1: return store(r[3], r[0], r[1], r[2]);
    case 2: return store(r[2], r[3], r[0], r[1]);
    default: return store(r[1], r[2], r[3], r[0]);
  }
}

// One wave per expert and token (blockIdx.y); blocks past the experts
// quantize the token's row.
template <typename TW>
__global__ __launch_bounds__(256) void route_rows_kernel(const RouteArgs a, int8_t *__restrict__ qx,
                                                         float *__restrict__ sx) {
  const int lane = threadIdx.x & 63;
  const int e = blockIdx.x * 4 + (threadIdx.x >> 6), m = blockIdx.y;
  if ((int)blockIdx.x >= (a.E + 3) / 4) return quant_row<256>(a, m, qx, sx);
  if (e >= a.E) return;
  const TW *w = static_cast<const TW *>(a.Wr) + (size_t)e * a.K;
  const float *x = a.X + (size_t)m * a.K;
  double acc = 0.;
#pragma unroll 8
  for (int k = 4 * lane; k < a.K; k += 256) {
    double wv[4], xv[4];
    load4(w + k, wv);
    load4(x + k, xv);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc = fma(xv[i], wv[i], acc);
  }
  const double s = wave_sum_f64(acc);
  if (lane == 0) a.logits[(size_t)m * a.E + e] = s;
}

template <int NE>
__global__ __launch_bounds__(256) void route_choice_kernel(const RouteArgs a) {
  const int lane = threadIdx.x & 63;
  const int m = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (m >= a.M) return;
  int id;
  float w;
  choose<NE>(a, a.logits + (size_t)m * a.E, lane, true, id, w);
  if (lane < a.top_k) {
    a.ids[(size_t)m * a.top_k + lane] = id;
    a.weights[(size_t)m * a.top_k + lane] = w;
  }
}

// Several partial sums: a workgroup per token adds them in increasing order
// (a thread per expert, four loads at a time), its first wave chooses.
template <int NE>
__global__ __launch_bounds__(256) void route_sum_choice_kernel(const RouteArgs a) {
  __shared__ double l[64 * NE];
  const int m = blockIdx.x;
  const size_t step = (size_t)a.M * a.E;
  for (int e = threadIdx.x; e < a.E; e += 256) {
    const double *p = a.logits + (size_t)m * a.E + e;
    double v = p[0];
    int k = 1;
    for (; k + 4 <= a.KS; k += 4) {
      const double p0 = p[k * step], p1 = p[(k + 1) * step], p2 = p[(k + 2) * step], p3 = p[(k + 3) * step];
      v = (((v + p0) + p1) + p2) + p3;
    }
    for (; k < a.KS; ++k) v += p[k * step];
    l[e] = v;
  }
  __syncthreads();
  if (threadIdx.x >= 64) return;
  int id;
  float w;
  choose<NE>(a, l, threadIdx.x, true, id, w);
  if ((int)threadIdx.x < a.top_k) {
    a.ids[(size_t)m * a.top_k + threadIdx.x] = id;
    a.weights[(size_t)m * a.top_k + threadIdx.x] = w;
  }
}

template <int NE>
void launch_choice(const RouteArgs &a, hipStream_t stream) {
  if (a.KS > 1) hipLaunchKernelGGL(route_sum_choice_kernel<NE>, dim3(a.M), dim3(256), 0, stream, a);
  else hipLaunchKernelGGL(route_choice_kernel<NE>, dim3((a.M + 3) / 4), dim3(256), 0, stream, a);
}

// qx, sx: also quantize X (or nullptr).
template <typename TW>
hipError_t launch_logits(const RouteArgs &a, int8_t *qx, float *sx, hipStream_t stream) {
  if (route_by_rows(a.M, a.E)) {
    hipLaunchKernelGGL(route_rows_kernel<TW>, dim3((a.E + 3) / 4 + (qx ? 1 : 0), a.M), dim3(256), 0, stream, a, qx, sx);
  } else {
    const int tiles = ((a.M + 31) / 32) * ((a.E + 31) / 32) * a.KS;
    hipLaunchKernelGGL(route_tile_kernel<TW>, dim3(tiles + (qx ? a.M : 0)), dim3(256), 0, stream, a, qx, sx);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route_front(const RouteArgs &a, int8_t *qx, float *sx, hipStream_t stream) {
  return a.wr_type == AQ_TYPE_F32 ? launch_logits<float>(a, qx, sx, stream)
                                  : launch_logits<uint16_t>(a, qx, sx, stream);
}

hipError_t launch_route_choice(const RouteArgs &a, hipStream_t stream) {
  if (a.E <= 64) launch_choice<1>(a, stream);
  else if (a.E <= 128) launch_choice<2>(a, stream);
  else if (a.E <= 256) launch_choice<4>(a, stream);
  else launch_choice<16>(a, stream);
  return hipGetLastError();
}

hipError_t launch_route(const RouteArgs &a, hipStream_t stream) {
  const hipError_t e = launch_route_front(a, nullptr, nullptr, stream);
  return e != hipSuccess ? e : launch_route_choice(a, stream);
}

}  // namespace aq
