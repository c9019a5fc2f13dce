// Attention over the 4-bit cache for few query rows (single tokens, short
// chunks): bound by the cache's bytes.
//
// A workgroup takes 16 rows of one sequence and key/value head and a range of
// its keys; its four waves take 32 keys each in turn and meet at the end.  A
// wave forms S^T = K Q^T (16 keys x 16 rows a tile), whose registers are, as
// they stand, the weights' operand of O^T = V^T P^T: the order of the keys in
// that product is free, and the values' codes are loaded in the order that the
// weights have.  So nothing passes through LDS but the waves' sums at the end,
// and the codes widen in registers (aq_attn.h).
//
// Long contexts are cut into ranges, a workgroup each, whose sums a second
// launch joins.

#include "aq_attn.h"

namespace aq {
namespace {

constexpr int kRows = 16, kUnit = 128;  // rows a workgroup; keys its waves take in a turn

// What a wave holds of 32 keys (two tiles of 16).
template <int D>
struct Keys {
  uint32_t k[2][D / 32];  // this lane's D/4 features of key lane % 16
  uint32_t v[8];          // D/16 features of keys 4g .. 4g+3 of both tiles
  u4 wk[2], wv[2];        // words of keys 4g .. 4g+3
  uint32_t wz[2];         // word of key lane % 16
};

template <int D>
__device__ __forceinline__ void load_tile(const AttnArgs &a, int head, int page, int tok, int t, Keys<D> &x) {
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const size_t vec = (((size_t)page * 2 * a.c.heads + head) << a.c.shift) + tok;
  const size_t val = (size_t)a.c.heads << a.c.shift;  // vectors from a page's keys to its values
  const uint8_t *k = a.c.codes + vec * (D / 2) + col * (D / 2) + g * (D / 8);
  if constexpr (D == 128) {
    const u4 w = *reinterpret_cast<const u4 *>(k);
    x.k[t][0] = w.x; x.k[t][1] = w.y; x.k[t][2] = w.z; x.k[t][3] = w.w;
  } else {
    const u2 w = *reinterpret_cast<const u2 *>(k);
    x.k[t][0] = w.x; x.k[t][1] = w.y;
  }
  const uint8_t *v = a.c.codes + (vec + val) * (D / 2) + (4 * g) * (D / 2) + col * (D / 32);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x.v[4 * t + i] = D == 128 ? *reinterpret_cast<const uint32_t *>(v + i * (D / 2))
                              : *reinterpret_cast<const uint16_t *>(v + i * (D / 2));
  x.wk[t] = *reinterpret_cast<const u4 *>(a.c.words + vec + 4 * g);
  x.wv[t] = *reinterpret_cast<const u4 *>(a.c.words + vec + val + 4 * g);
  x.wz[t] = a.c.words[vec + col];
}

template <int D>
__global__ __launch_bounds__(256) void attn_rows_kernel(AttnArgs a) {
  constexpr int KS = D / 32, DT = D / 16;
  constexpr int LD = D + 4;
  __shared__ float so[4][kRows][LD];
  __shared__ float sm[4][kRows], sl[4][kRows];
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int tile = blockIdx.x / a.c.heads, head = blockIdx.x - tile * a.c.heads, split = blockIdx.y;
  Rows r;
  if (!find_rows<kRows>(a, tile, r)) return;
  const int before = r.len - r.n;  // keys in front of the sequence's first query
  const int row = min(r.r0 + col, r.rows - 1), last = min(r.r0 + kRows, r.rows) - 1;
  const int vis = before + row / a.G + 1;  // keys that this lane's row sees
  const int limit = max(0, before + last / a.G + 1), all = before + r.r0 / a.G + 1;
  const Range kr = split_range(limit, kUnit, a.splits, split);
  if (split >= kr.ranges) return;

  // q in two pieces
  h8 qh[KS], ql[KS];
  float rf;
  {
    const float *q = a.q + (size_t)(r.first + row / a.G) * a.ldq + (size_t)(head * a.G + row % a.G) * D + g * (D / 4);
    float x[KS][8], amax = 0.f;
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(q + 8 * s + j);
        x[s][j] = v.x; x[s][j + 1] = v.y; x[s][j + 2] = v.z; x[s][j + 3] = v.w;
        amax = fmaxf(amax, fmaxf(fmaxf(finite_abs(v.x), finite_abs(v.y)), fmaxf(finite_abs(v.z), finite_abs(v.w))));
      }
    amax = fmaxf(amax, __shfl_xor(amax, 16));
    amax = fmaxf(amax, __shfl_xor(amax, 32));
    float up, down;
    row_factor(amax, up, down);
    rf = down * a.scale;
#pragma unroll
    for (int s = 0; s < KS; ++s) pieces8(x[s], up, qh[s], ql[s]);
  }

  f4 o[DT];
#pragma unroll
  for (int j = 0; j < DT; ++j) o[j] = f4{0.f, 0.f, 0.f, 0.f};
  float M = kNone, l = 0.f;

  // Page ids of 32 turns at a time, lane 2j + t that of tile t in turn j; -1
  // where no key is visible or the table has no page.
  const int32_t *table = a.table + (size_t)r.b * a.width;
  const int mask = (1 << a.c.shift) - 1;
  int ids = -1, u_ids = kr.u0 - 32;
  auto pages = [&](int u) {
    if (u - u_ids >= 32) {
      u_ids = u;
      const int key = (u + (lane >> 1)) * kUnit + wave * 32 + 16 * (lane & 1);
      ids = -1;
      if (key >= 0 && key < limit) ids = table[key >> a.c.shift];
      if ((unsigned)ids >= (unsigned)a.c.pages) ids = -1;
    }
  };
  auto load = [&](int u, Keys<D> &x, int (&id)[2]) {
    pages(u);
    const int key0 = u * kUnit + wave * 32;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      id[t] = __builtin_amdgcn_readlane(ids, 2 * (u - u_ids) + t);
      load_tile<D>(a, head, max(id[t], 0), (key0 + 16 * t) & mask, t, x);
    }
  };

  Keys<D> x;
  int id[2] = {-1, -1};
  if (kr.u0 < kr.u1) load(kr.u0, x, id);
  for (int u = kr.u0; u < kr.u1; ++u) {
    Keys<D> y;
    int idy[2] = {-1, -1};
    if (u + 1 < kr.u1) load(u + 1, y, idy);
    if (id[0] >= 0 || id[1] >= 0) {
      const int key0 = u * kUnit + wave * 32;
      // scores
      float s[8], wv[8];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const Zero z = zero_of(x.wz[t] & 15u, x.wz[t] & 15u);
        f4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          const h8 kf = widen8(x.k[t][j], z);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qh[j], acc, 0, 0, 0);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, ql[j], acc, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s[4 * t + i] = fmaf(acc[i] * scale_of(x.wk[t][i]), rf, exp_of(x.wv[t][i]));
      }
      const bool full = id[0] >= 0 && id[1] >= 0 && key0 + 32 <= all;
      if (!full) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int key = key0 + 16 * (e >> 2) + 4 * g + (e & 3);
          if (id[e >> 2] < 0 || key >= vis) s[e] = -__builtin_inff();
        }
      }
      float top = fmaxf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])), fmaxf(fmaxf(s[4], s[5]), fmaxf(s[6], s[7])));
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      if (__any(top > M)) {
        const float up = fmaxf(M, top), f = exp2_fast(M - up);
        M = up;
        l *= f;
#pragma unroll
        for (int j = 0; j < DT; ++j) o[j] *= f;
      }
      // weights
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t w = x.wv[e >> 2][e & 3];
        const float p = exp2_fast(s[e] - M);
        float d = p * inv_exp_of(w);
        wv[e] = p * frac_of(w);
        if (!full) {
          const int key = key0 + 16 * (e >> 2) + 4 * g + (e & 3);
          const bool ok = id[e >> 2] >= 0 && key < vis;
          d = ok ? d : 0.f;
          wv[e] = ok ? wv[e] : 0.f;
        }
        l += d;
      }
      h8 ph, pl;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        _Float16 hi, lo;
        pieces(wv[e], hi, lo);
        ph[e] = hi;
        pl[e] = lo;
      }
      // values: byte b of the tokens' words holds features 2b and 2b + 1
      Zero z[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) z[p] = zero_of(x.wv[p >> 1][2 * (p & 1)] & 15u, x.wv[p >> 1][2 * (p & 1) + 1] & 15u);
#pragma unroll
      for (int b = 0; b < DT / 2; ++b) {
        h8 lo, hi;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t two = __builtin_amdgcn_perm(x.v[2 * p + 1], x.v[2 * p], 0x0C040C00u + 0x00010001u * b);
          const h2 c = widen_lo(two, z[p]), d = widen_hi(two, z[p]);
          lo[2 * p] = c.x; lo[2 * p + 1] = c.y;
          hi[2 * p] = d.x; hi[2 * p + 1] = d.y;
        }
        o[2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(lo, ph, o[2 * b], 0, 0, 0);
        o[2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(lo, pl, o[2 * b], 0, 0, 0);
        o[2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(hi, ph, o[2 * b + 1], 0, 0, 0);
        o[2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(hi, pl, o[2 * b + 1], 0, 0, 0);
      }
    }
    x = y;
    id[0] = idy[0];
    id[1] = idy[1];
  }

  // the four waves' sums
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (g == 0) {
    sm[wave][col] = M;
    sl[wave][col] = l;
  }
  __syncthreads();
  const float top = fmaxf(fmaxf(sm[0][col], sm[1][col]), fmaxf(sm[2][col], sm[3][col]));
  const float f = exp2_fast(M - top);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < DT; ++j) so[wave][col][DT * (4 * g + i) + j] = o[j][i] * f;
  __syncthreads();
  const int here = last - r.r0 + 1;
  for (int e = threadIdx.x; e < here * (D / 4); e += 256) {
    const int rr = e / (D / 4), d = 4 * (e % (D / 4));
    f4 v = {0.f, 0.f, 0.f, 0.f};
    float m = sm[0][rr], sum = 0.f;
#pragma unroll
    for (int w = 1; w < 4; ++w) m = fmaxf(m, sm[w][rr]);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      v += *reinterpret_cast<const f4 *>(&so[w][rr][d]);
      sum += sl[w][rr] * exp2_fast(sm[w][rr] - m);
    }
    const int rw = r.r0 + rr;
    if (kr.ranges == 1) {
      v *= inv_sum(sum) * (1.f / (1 << kPieceBias));
      *reinterpret_cast<f4 *>(a.out + ((size_t)(r.first + rw / a.G) * a.Hq + head * a.G + rw % a.G) * D + d) = v;
    } else {
      const size_t at = (((size_t)split * a.tiles + tile) * a.c.heads + head) * kRows + rr;
      float *part = a.part + at * (D + 4);
      *reinterpret_cast<f4 *>(part + d) = v;
      if (d == 0) {
        part[D] = m;
        part[D + 1] = sum;
      }
    }
  }
}

// The ranges' sums of a row joined: a wave per row, lane t first holding range t.
template <int D, int T>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, int unit) {
  constexpr int V = D / 64;
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int tile = blockIdx.x / a.c.heads, head = blockIdx.x - tile * a.c.heads;
  Rows r;
  if (!find_rows<T>(a, tile, r)) return;
  const int last = min(r.r0 + T, r.rows) - 1;
  const int limit = max(0, r.len - r.n + last / a.G + 1);
  const int ranges = split_range(limit, unit, a.splits, 0).ranges;
  if (ranges == 1) return;
  const size_t step = (size_t)a.tiles * a.c.heads * T * (D + 4);
  for (int rr = blockIdx.y * 4 + wave; rr <= last - r.r0; rr += 4 * gridDim.y) {
    const float *part = a.part + (((size_t)tile * a.c.heads + head) * T + rr) * (D + 4);
    float m = kNone, s = 0.f;
    if (lane < ranges) {
      m = part[lane * step + D];
      s = part[lane * step + D + 1];
    }
    float top = m;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
    const float f = exp2_fast(m - top);
    float sum = s * f;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o);
    float v[V] = {};
    for (int t = 0; t < ranges; ++t) {
      const float ft = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), t));
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += ft * part[t * step + V * lane + i];
    }
    const float n = inv_sum(sum) * (1.f / (1 << kPieceBias));
    const int rw = r.r0 + rr;
    float *out = a.out + ((size_t)(r.first + rw / a.G) * a.Hq + head * a.G + rw % a.G) * D + V * lane;
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = v[i] * n;
  }
}

template <int D, int T>
void join(const AttnArgs &a, int unit, hipStream_t stream) {
  // 16 rows a workgroup and more than that side by side
  hipLaunchKernelGGL((attn_join_kernel<D, T>), dim3((unsigned)(a.tiles * a.c.heads), (T + 15) / 16), dim3(256), 0, stream, a,
                     unit);
}

}  // namespace

hipError_t launch_attn_join(const AttnArgs &a, int rows, int unit, hipStream_t stream) {
  if (a.c.D == 128) {
    if (rows == 16) join<128, 16>(a, unit, stream);
    else join<128, 128>(a, unit, stream);
  } else {
    if (rows == 16) join<64, 16>(a, unit, stream);
    else join<64, 128>(a, unit, stream);
  }
  return hipGetLastError();
}

hipError_t launch_attn_rows(const AttnArgs &a, hipStream_t stream) {
  const dim3 g((unsigned)(a.tiles * a.c.heads), a.splits), b(256);
  if (a.c.D == 128)
    hipLaunchKernelGGL(attn_rows_kernel<128>, g, b, 0, stream, a);
  else
    hipLaunchKernelGGL(attn_rows_kernel<64>, g, b, 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  return launch_attn_join(a, kRows, kUnit, stream);
}

}  // namespace aq
