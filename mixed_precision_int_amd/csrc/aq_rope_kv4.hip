// Rotary positions with the append to the 4-bit cache (aq_rope_kv4), and the
// cache read back (aq_kv4_read).
//
// A wave takes a token and some of its heads; lane i holds one pair of a head's
// features (two heads side by side where D = 64), so that the angle of a lane,
// its sine and cosine, formed in FP64 for far positions, serve every head.  The
// turned value is rounded to FP32 once, from FP64: the codes of keys next to a
// tie are the definition's.

#include "aq_kv4.h"
#include "aq_layer.h"
#include "aq_quant.h"

namespace aq {
namespace {

constexpr int kWaves = 4;

// Maximum over 64 (D = 128) or each 32 lanes (D = 64), of values at least 0 (as bits
// their order is that of whole numbers): DPP within rows of 16, then across them.
template <int D>
__device__ __forceinline__ float heads_max(float x) {
  uint32_t v = __float_as_uint(x);
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
  const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(p[0], p[1]);
  if constexpr (D == 128) {
    const auto q = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max(q[0], q[1]);
  }
  return __uint_as_float(v);
}

// rint(x / s) + z, clipped: the FP32 quotient p = x * fl32(1/s) decides unless
// it is near a tie (|x / s| <= 15, so |p - x / s| < 2^-18 where |p| <= 16).
__device__ __forceinline__ int code4(float x, double s, float inv, double z) {
  const float p = x * inv, r = rintf(p);
  double q = r;
  if (!(fabsf(p - r) < 0.5f - 0x1p-15f && fabsf(r) <= 16.f)) q = rint((double)x / s);
  q += z;
  return (int)fmin(fmax(q, 0.), 15.);
}

// A head's vector (two features of it in each of D/2 lanes) into the cache.
// `held` is uniform over the head's lanes; nib is D bytes of LDS of its own.
template <int D>
__device__ __forceinline__ void hold(float x, float y, int fx, int fy, bool held, uint8_t *row, uint32_t *word,
                                     uint8_t *nib) {
  const int lane = threadIdx.x & (D / 2 - 1);
  const bool odd = !(fabsf(x) <= 3.402823466e38f && fabsf(y) <= 3.402823466e38f);
  const uint64_t all = __ballot(odd);
  const bool bad = D == 128 ? all != 0 : (threadIdx.x & 32) ? (all >> 32) != 0 : (uint32_t)all != 0;
  const float hi = heads_max<D>(fmaxf(fmaxf(x, y), 0.f)), lo = -heads_max<D>(fmaxf(fmaxf(-x, -y), 0.f));
  const double want = fmax(((double)hi - (double)lo) / 15., 1e-12);
  float up = (float)want;
  uint32_t bits = __float_as_uint(up) + ((double)up < want ? 1u : 0u);
  bits = (bits + 15u) & ~15u;
  const bool none = bad || bits >= kNoScale;
  const double s = (double)__uint_as_float(bits);
  const double z = rint(-(double)lo / s);
  const float inv = (float)(1. / s);
  nib[fx] = none ? 0 : (uint8_t)code4(x, s, inv, z);
  nib[fy] = none ? 0 : (uint8_t)code4(y, s, inv, z);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (held) {
    if (lane < D / 8) {
      const uint32_t *n = reinterpret_cast<const uint32_t *>(nib) + 2 * lane;
      const uint32_t a = n[0], b = n[1];
      // 8 features, a nibble each
      uint32_t w = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) w |= ((a >> (8 * i)) & 15u) << (4 * i) | ((b >> (8 * i)) & 15u) << (16 + 4 * i);
      reinterpret_cast<uint32_t *>(row)[lane] = w;
    }
    if (lane == 0) *word = none ? kNaNWord : bits | (uint32_t)(int)z;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <int D>
__global__ __launch_bounds__(64 * kWaves) void rope_kv4_kernel(RopeArgs a, int parts) {
  constexpr int HW = 128 / D;  // heads a wave holds at a time
  __shared__ alignas(16) uint8_t nibs[kWaves][128];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, i = lane & (D / 2 - 1), sub = lane / (D / 2);
  const long long unit = (long long)blockIdx.x * kWaves + wave;
  if (unit >= (long long)a.M * parts) return;
  const int m = (int)(unit / parts), part = (int)(unit % parts);
  const float *row = a.qkv + (size_t)m * a.ldqkv;
  float *qrow = a.Q + (size_t)m * a.ldq;
  const int heads = a.c.heads, all = a.Hq + 2 * heads;

  // this lane's pair of features
  int fx, fy;
  if (a.interleaved) {
    fx = 2 * i;
    fy = 2 * i + 1;
  } else if (i < a.pairs) {
    fx = i;
    fy = i + a.pairs;
  } else {
    fx = a.pairs + i;
    fy = D / 2 + i;
  }
  double sn = 0., cs = 1.;
  if (i < a.pairs) {
    int axis = 0;
#pragma unroll
    for (int t = 0; t + 1 < AQ_ROPE_MAX_AXES; ++t) axis += i >= a.end[t];
    const double angle = (double)a.pos[(size_t)axis * a.M + m] * (double)a.freq[i];
    sincos(angle, &sn, &cs);
  }
  const long long slot = a.slots[m];
  const bool in = slot >= 0 && slot < ((long long)a.c.pages << a.c.shift);
  const size_t page = in ? (size_t)(slot >> a.c.shift) : 0;
  const int tok = in ? (int)(slot & ((1 << a.c.shift) - 1)) : 0;

  // Eight heads' loads at a time: with one, a token's heads are a chain of round trips to
  // memory.
  constexpr int U = 8;
  const int step = parts * HW;
  for (int h0 = part * HW; h0 < all; h0 += U * step) {
    float x[U], y[U];
#pragma unroll
    for (int t = 0; t < U; ++t) {
      const int h = min(h0 + t * step + sub, all - 1);
      x[t] = row[(uint32_t)(h * D + fx)];
      y[t] = row[(uint32_t)(h * D + fy)];
    }
#pragma unroll
    for (int t = 0; t < U; ++t) {
      const int first = h0 + t * step, h = first + sub;
      if (first >= all) break;
      if (h < a.Hq + heads && i < a.pairs) {
        const double p = x[t], q = y[t];
        x[t] = (float)(p * cs - q * sn);
        y[t] = (float)(q * cs + p * sn);
      }
      if (h < a.Hq) {
        qrow[(uint32_t)(h * D + fx)] = x[t];
        qrow[(uint32_t)(h * D + fy)] = y[t];
      }
      if (first + HW > a.Hq) {  // (wave-uniform) some head of the wave is a key or a value
        const bool key = h < a.Hq + heads;
        const int kv = key ? 0 : 1, hh = h - a.Hq - (key ? 0 : heads);
        const bool held = in && h < all && h >= a.Hq;
        const size_t at = held ? (((page * 2 + kv) * heads + hh) << a.c.shift) + tok : 0;
        hold<D>(x[t], y[t], fx, fy, held, a.c.codes + at * (D / 2), a.c.words + at, nibs[wave] + sub * D);
      }
    }
  }
}

template <int D>
__global__ __launch_bounds__(256) void kv4_read_kernel(Kv4View c, const int64_t *slots, int M, float *K, float *V, uint32_t first) {
  constexpr int L = D / 8;  // lanes a vector, 8 features each
  const uint64_t t = (uint64_t)first * 256 + (uint64_t)blockIdx.x * 256 + threadIdx.x;
  const long long vec = (long long)(t / L);
  const int part = (int)(t % L);
  if (vec >= (long long)M * 2 * c.heads) return;
  const int h = (int)(vec % c.heads), kv = (int)(vec / c.heads % 2), m = (int)(vec / c.heads / 2);
  const long long slot = slots[m];
  float x[8] = {};
  if (slot >= 0 && slot < ((long long)c.pages << c.shift)) {
    const size_t at = ((((size_t)(slot >> c.shift) * 2 + kv) * c.heads + h) << c.shift) + (slot & ((1 << c.shift) - 1));
    const uint32_t w = c.words[at], b = reinterpret_cast<const uint32_t *>(c.codes + at * (D / 2))[part];
    const float s = scale_held(w);
    const int z = (int)(w & 15u);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = s * (float)((int)(b >> (4 * i) & 15u) - z);
  }
  float4 *out = reinterpret_cast<float4 *>((kv ? V : K) + ((size_t)m * c.heads + h) * D + 8 * part);
  out[0] = make_float4(x[0], x[1], x[2], x[3]);
  out[1] = make_float4(x[4], x[5], x[6], x[7]);
}

}  // namespace

hipError_t launch_rope_kv4(const RopeArgs &a, hipStream_t stream) {
  // A wave of a token computes its sines once, so more waves per token cost more of them;
  // fewer leave the memory idle.  5000 tokens of 56 heads (251 MB, a copy of which takes 52 us):
  // 78 us with one wave per token and a head's loads at a time, 61 with four heads', 51
  // with four waves per token and eight heads' (52 with eight waves, 56 with two).
  const int steps = (a.Hq + 2 * a.c.heads + 128 / a.c.D - 1) / (128 / a.c.D);
  int parts = 1;
  while (parts < 16 && parts * 2 <= steps && (long long)a.M * parts < 16384) parts *= 2;
  const dim3 g((unsigned)(((long long)a.M * parts + kWaves - 1) / kWaves)), b(64 * kWaves);
  if (a.c.D == 128)
    hipLaunchKernelGGL(rope_kv4_kernel<128>, g, b, 0, stream, a, parts);
  else
    hipLaunchKernelGGL(rope_kv4_kernel<64>, g, b, 0, stream, a, parts);
  return hipGetLastError();
}

hipError_t launch_kv4_read(const Kv4View &c, const int64_t *slots, int M, float *K, float *V, hipStream_t stream) {
  const long long threads = (long long)M * 2 * c.heads * (c.D / 8);
  // (a launch has less than 2^32 threads)
  constexpr long long kMost = 1 << 23;
  for (long long first = 0, n = (threads + 255) / 256; first < n; first += kMost) {
    const dim3 g((unsigned)(n - first < kMost ? n - first : kMost)), b(256);
    if (c.D == 128)
      hipLaunchKernelGGL(kv4_read_kernel<128>, g, b, 0, stream, c, slots, M, K, V, (uint32_t)first);
    else
      hipLaunchKernelGGL(kv4_read_kernel<64>, g, b, 0, stream, c, slots, M, K, V, (uint32_t)first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace aq
