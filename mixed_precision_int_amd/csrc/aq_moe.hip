// A mixture-of-experts layer for a few tokens over packed W4/W8 experts.
//
// For each pair (token m, slot i) with expert e = ids[m][i]:
//   g, u = s_x sum_j S[n,j] P[m,n,j]   over the expert's gate and up rows
//   h    = fl32( g / (1 + exp(-g)) * u )
//   qh, sh = the per-token INT8 quantizer over h's row
//   y[m] = sum_i w[m][i] sh sum_j S2[n,j] P2[pair,n,j]
// P the INT32 tile products (AlignQuant eq. 19), S the FP32 row scales.
//
// g and u are summed in FP64 (the products P S have at most 45 bits, so each
// is exact) and h is rounded once: the codes qh then equal those of the
// definition.  With FP32 sums about one row in five would hold a code that
// is off by one, which moves the row's outputs by some 1e-3.  The down
// projection's sums feed no quantizer and stay in FP32.
//
// Work: the pairs are grouped by expert, so that an expert's weights are
// read once for up to 16 of its tokens (one MFMA operand).

#include "aq_device.h"
#include "aq_routed.h"

namespace aq {
namespace {

__device__ __forceinline__ v4i load16(const void *p) { return *reinterpret_cast<const v4i *>(p); }

// Packed projection as the kernels read it.
struct Packed {
  const uint8_t *labels;
  const int32_t *off4, *off8;
  const uint8_t *w4;
  const uint8_t *w8;
  const float *s4, *s8;
  int C, K, T4, T8, label_words;
};
Packed packed_of(const PackedView &v) {
  Packed p;
  p.labels = v.labels; p.off4 = v.off4; p.off8 = v.off8;
  p.w4 = v.w4; p.w8 = reinterpret_cast<const uint8_t *>(v.w8);
  p.s4 = v.s4; p.s8 = v.s8;
  p.C = v.C; p.K = v.K; p.T4 = v.T4; p.T8 = v.T8;
  p.label_words = (int)(((long long)v.R * v.C + 31) / 32);
  return p;
}

// One lane's share of a 16-row group of one tile: row i16 (rowoff: its bytes
// inside a 1 KB panel), k-group g.
struct TileW {
  v4i a, b;
  float sc;       // row scale, with the 1/16 of the INT4 widening
  int is4, live;
};

// Walks the tiles of one tile row from column c0 on (eq. 16 indices).
struct RowWalk {
  int tb, idx4, idx8;
  __device__ __forceinline__ RowWalk(const Packed &p, int r, int c0) {
    tb = r * p.C;
    const int n4 = count_int4(p.labels, tb, c0, p.label_words);
    idx4 = p.off4[r] + n4;
    idx8 = p.off8[r] + (c0 - n4);
  }
};

// Loads tile column j (walked in increasing order).  Inconsistent metadata
// (an index outside the buffers) makes the tile a dead one.
template <int BK>
__device__ __forceinline__ void load_tile(const Packed &p, RowWalk &w, int j, uint32_t labs, int g, int rowoff,
                                          TileW &t) {
  const int is4 = (int)(labs & 1u);
  const int idx = is4 ? w.idx4 : w.idx8;
  w.idx4 += is4;
  w.idx8 += is4 ^ 1;
  t.is4 = is4;
  t.live = idx >= 0 && idx < (is4 ? p.T4 : p.T8);
  if (!t.live) return;
  if (BK == 128) {
    if (is4) {
      t.a = load16(p.w4 + (size_t)idx * 4096 + g * 1024 + rowoff);
    } else {
      const uint8_t *b = p.w8 + (size_t)idx * 8192 + 2 * g * 1024 + rowoff;
      t.a = load16(b);
      t.b = load16(b + 1024);
    }
  } else if (is4) {
    const uint2 lo = *reinterpret_cast<const uint2 *>(p.w4 + (size_t)idx * 2048 + (g >> 1) * 1024 + rowoff + 8 * (g & 1));
    t.a = v4i{(int)lo.x, (int)lo.y, 0, 0};
  } else {
    t.a = load16(p.w8 + (size_t)idx * 4096 + g * 1024 + rowoff);
  }
  t.sc = (is4 ? p.s4 : p.s8)[(size_t)idx * 64 + (rowoff >> 4)];
}

// INT32 product of the tile with 16 token rows; x points at the lane's token
// row, column j * BK.  INT4 codes are widened x16 (exact; undone by sc).
template <int BK>
__device__ __forceinline__ v4i tile_product(const TileW &t, const int8_t *x, int g) {
  v4i acc = {0, 0, 0, 0};
  if (BK == 128) {
    const v4i x0 = load16(x + 32 * g), x1 = load16(x + 32 * g + 16);
    v4i w0 = t.a, w1 = t.b;
    if (t.is4) {
      w0 = v4i{w4_lo16(t.a[0]), w4_lo16(t.a[1]), w4_lo16(t.a[2]), w4_lo16(t.a[3])};
      w1 = v4i{w4_hi16(t.a[0]), w4_hi16(t.a[1]), w4_hi16(t.a[2]), w4_hi16(t.a[3])};
    }
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(x0, w0, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(x1, w1, acc, 0, 0, 0);
  } else {
    v4i xo, w0 = t.a;
    if (t.is4) {
      const int8_t *c = x + 32 * (g >> 1) + 8 * (g & 1);
      const uint2 p0 = *reinterpret_cast<const uint2 *>(c), p1 = *reinterpret_cast<const uint2 *>(c + 16);
      xo = v4i{(int)p0.x, (int)p0.y, (int)p1.x, (int)p1.y};
      w0 = v4i{w4_lo16(t.a[0]), w4_lo16(t.a[1]), w4_hi16(t.a[0]), w4_hi16(t.a[1])};
    } else {
      xo = load16(x + 16 * g);
    }
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(xo, w0, acc, 0, 0, 0);
  }
  return acc;
}

// ---- lists: pairs grouped by expert.  lists[0] = number of active experts,
// then active [E], start [E + 1], pair [P].  One workgroup; an id outside
// 0 .. E-1 belongs to no expert.  The place of a pair inside its expert's
// run depends on the order of the LDS atomics, its result does not: every
// pair is one row of an MFMA operand and its outputs are its own.
constexpr int kMoeMaxE = 1024;
__global__ __launch_bounds__(1024) void moe_lists_kernel(const int32_t *__restrict__ ids, int P, int E,
                                                         int32_t *__restrict__ lists) {
  __shared__ int cnt[kMoeMaxE], pos[kMoeMaxE];
  __shared__ int wsum[16], wact[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  cnt[tid] = 0;
  __syncthreads();
  for (int p = tid; p < P; p += 1024) {
    const int e = ids[p];
    if ((unsigned)e < (unsigned)E) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  // exclusive scans over the experts: pairs before, active experts before
  const int c = tid < E ? cnt[tid] : 0;
  int s = c, a = c > 0;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int ps = __shfl_up(s, o), pa = __shfl_up(a, o);
    if (lane >= o) {
      s += ps;
      a += pa;
    }
  }
  if (lane == 63) {
    wsum[wave] = s;
    wact[wave] = a;
  }
  __syncthreads();
  for (int w = 0; w < wave; ++w) {
    s += wsum[w];
    a += wact[w];
  }
  int32_t *active = lists + 1, *start = active + E, *pair = start + E + 1;
  if (tid < E) {
    start[tid] = s - c;
    pos[tid] = s - c;
    if (c > 0) active[a - 1] = tid;
  }
  if (tid == 1023) {
    lists[0] = a;
    start[E] = s;
  }
  __syncthreads();
  for (int p = tid; p < P; p += 1024) {
    const int e = ids[p];
    if ((unsigned)e < (unsigned)E) pair[atomicAdd(&pos[e], 1)] = p;
  }
}

struct MoeArgs {
  Packed gu, dn;
  const int8_t *qx;
  const float *sx;
  const int32_t *ids;
  const float *weights;
  const int32_t *lists;
  float *h;
  int8_t *qh;
  float *sh;
  float *d;
  float *Y;
  int M, top_k, E, H, I;
};

// ---- gate and up: one workgroup per 16 features of one active expert (its
// 16 gate rows and 16 up rows); the waves cut the tile columns, their FP64
// sums meet in LDS in increasing order.
constexpr int kGuWaves = 8;
constexpr int kGuDepth = 2;  // tile columns per load batch

template <int BK>
__global__ __launch_bounds__(kGuWaves * 64) void moe_gate_up_kernel(const MoeArgs a) {
  __shared__ double red[kGuWaves][2][4][64];
  if ((int)blockIdx.y >= a.lists[0]) return;
  const int e = a.lists[1 + blockIdx.y];
  const int32_t *start = a.lists + 1 + a.E;
  const int p0 = start[e], cnt = start[e + 1] - p0;
  const int32_t *pair = start + a.E + 1 + p0;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  const int t = blockIdx.x >> 2, rg = blockIdx.x & 3;
  const int rowoff = rg * 256 + i16 * 16;
  const int C = a.gu.C, RI = a.I >> 6;
  const int c0 = C * wave / kGuWaves, c1 = C * (wave + 1) / kGuWaves;
  const int rgate = e * 2 * RI + t;
  for (int b = 0; b < cnt; b += 16) {
    const int pr = pair[min(b + i16, cnt - 1)];  // tokens past the last repeat it; not stored
    const int8_t *x = a.qx + (size_t)(pr / a.top_k) * a.gu.K;
    RowWalk wg(a.gu, rgate, c0), wu(a.gu, rgate + RI, c0);
    double G[4] = {0., 0., 0., 0.}, U[4] = {0., 0., 0., 0.};
    for (int j0 = c0; j0 < c1; j0 += kGuDepth) {
      TileW tg[kGuDepth], tu[kGuDepth];
      const uint32_t lg = label_bits32(a.gu.labels, wg.tb + j0, a.gu.label_words);
      const uint32_t lu = label_bits32(a.gu.labels, wu.tb + j0, a.gu.label_words);
#pragma unroll
      for (int q = 0; q < kGuDepth; ++q) {
        tg[q].live = tu[q].live = 0;
        if (j0 + q < c1) {
          load_tile<BK>(a.gu, wg, j0 + q, lg >> q, g, rowoff, tg[q]);
          load_tile<BK>(a.gu, wu, j0 + q, lu >> q, g, rowoff, tu[q]);
        }
      }
#pragma unroll
      for (int q = 0; q < kGuDepth; ++q) {
        const int8_t *xc = x + (size_t)(j0 + q) * BK;
        if (tg[q].live) {
          const v4i p = tile_product<BK>(tg[q], xc, g);
          const double sc = (double)tg[q].sc * (tg[q].is4 ? 0.0625 : 1.0);
#pragma unroll
          for (int k = 0; k < 4; ++k) G[k] = fma((double)p[k], sc, G[k]);
        }
        if (tu[q].live) {
          const v4i p = tile_product<BK>(tu[q], xc, g);
          const double sc = (double)tu[q].sc * (tu[q].is4 ? 0.0625 : 1.0);
#pragma unroll
          for (int k = 0; k < 4; ++k) U[k] = fma((double)p[k], sc, U[k]);
        }
      }
    }
    if (b) __syncthreads();  // the last group's sums have been read
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      red[wave][0][k][lane] = G[k];
      red[wave][1][k][lane] = U[k];
    }
    __syncthreads();
    if (threadIdx.x < 256) {  // element k = wave of lane: token 4g + k, feature i16
      const int tok = b + 4 * g + wave;
      if (tok < cnt) {
        double sg = 0., su = 0.;
#pragma unroll
        for (int w = 0; w < kGuWaves; ++w) {
          sg += red[w][0][wave][lane];
          su += red[w][1][wave][lane];
        }
        const int p = pair[tok];
        const double s = (double)a.sx[p / a.top_k];
        sg *= s;
        su *= s;
        a.h[(size_t)p * a.I + (blockIdx.x << 4) + i16] = (float)(sg / (1. + exp(-sg)) * su);
      }
    }
  }
}

// ---- down: one workgroup per tile row of one active expert, 4 row groups x
// S column splits; the splits' FP32 sums are added in increasing order.
template <int BK, int S>
__global__ __launch_bounds__(S * 256) void moe_down_kernel(const MoeArgs a) {
  __shared__ float4 red[S > 1 ? S * 4 : 1][64];
  constexpr int DEPTH = 4;
  if ((int)blockIdx.y >= a.lists[0]) return;
  const int e = a.lists[1 + blockIdx.y];
  const int32_t *start = a.lists + 1 + a.E;
  const int p0 = start[e], cnt = start[e + 1] - p0;
  const int32_t *pair = start + a.E + 1 + p0;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  const int rg = wave & 3, sp = wave >> 2;
  const int rowoff = rg * 256 + i16 * 16;
  const int C = a.dn.C;
  const int c0 = C * sp / S, c1 = C * (sp + 1) / S;
  const int r = e * (a.H >> 6) + blockIdx.x;
  for (int b = 0; b < cnt; b += 16) {
    const int8_t *x = a.qh + (size_t)pair[min(b + i16, cnt - 1)] * a.I;
    RowWalk wk(a.dn, r, c0);
    float F[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = c0; j0 < c1; j0 += DEPTH) {
      TileW t[DEPTH];
      const uint32_t labs = label_bits32(a.dn.labels, wk.tb + j0, a.dn.label_words);
#pragma unroll
      for (int q = 0; q < DEPTH; ++q) {
        t[q].live = 0;
        if (j0 + q < c1) load_tile<BK>(a.dn, wk, j0 + q, labs >> q, g, rowoff, t[q]);
      }
#pragma unroll
      for (int q = 0; q < DEPTH; ++q) {
        if (t[q].live) {
          const v4i p = tile_product<BK>(t[q], x + (size_t)(j0 + q) * BK, g);
          const float sc = t[q].is4 ? t[q].sc * 0.0625f : t[q].sc;
#pragma unroll
          for (int k = 0; k < 4; ++k) F[k] = fmaf((float)p[k], sc, F[k]);
        }
      }
    }
    if (S > 1) {
      if (b) __syncthreads();
      red[wave][lane] = make_float4(F[0], F[1], F[2], F[3]);
      __syncthreads();
      if (sp == 0) {
#pragma unroll
        for (int s = 1; s < S; ++s) {
          const float4 v = red[4 * s + rg][lane];
          F[0] += v.x; F[1] += v.y; F[2] += v.z; F[3] += v.w;
        }
      }
    }
    if (sp == 0) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int tok = b + 4 * g + k;
        if (tok < cnt) {
          const int p = pair[tok];
          a.d[(size_t)p * a.H + blockIdx.x * 64 + rg * 16 + i16] = F[k] * a.sh[p] * a.weights[p];
        }
      }
    }
  }
}

// ---- combine: a token's outputs added in slot order.
__global__ __launch_bounds__(256) void moe_combine_kernel(const MoeArgs a) {
  const int m = blockIdx.y;
  const int n4 = a.H >> 2;
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= n4) return;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < a.top_k; ++i) {
    const size_t p = (size_t)m * a.top_k + i;
    if ((unsigned)a.ids[p] >= (unsigned)a.E) continue;
    const float4 v = reinterpret_cast<const float4 *>(a.d + p * a.H)[c];
    y.x += v.x; y.y += v.y; y.z += v.z; y.w += v.w;
  }
  reinterpret_cast<float4 *>(a.Y + (size_t)m * a.H)[c] = y;
}

// h rows of pairs that no expert computed are cleared for the quantizer,
// which runs over all pairs.
__global__ __launch_bounds__(256) void moe_clear_kernel(const MoeArgs a) {
  const size_t p = blockIdx.x;
  if ((unsigned)a.ids[p] < (unsigned)a.E) return;
  for (int i = threadIdx.x; i < a.I; i += 256) a.h[p * a.I + i] = 0.f;
}

}  // namespace

hipError_t launch_moe_experts(const MoeShape &s, const PackedView &gu, const PackedView &dn, const int8_t *qx,
                              const float *sx, const int32_t *ids, const float *weights, float *Y,
                              const MoeWs &ws, hipStream_t stream) {
  MoeArgs a;
  a.gu = packed_of(gu);
  a.dn = packed_of(dn);
  a.qx = qx; a.sx = sx; a.ids = ids; a.weights = weights; a.lists = ws.lists;
  a.h = ws.h; a.qh = ws.qh; a.sh = ws.sh; a.d = ws.d; a.Y = Y;
  a.M = s.M; a.top_k = s.top_k; a.E = s.E; a.H = s.H; a.I = s.I;
  const int P = s.pairs();
  const int slots = P < s.E ? P : s.E;
  hipError_t e;
  hipLaunchKernelGGL(moe_lists_kernel, dim3(1), dim3(1024), 0, stream, ids, P, s.E, ws.lists);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(moe_clear_kernel, dim3(P), dim3(256), 0, stream, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const dim3 g1(s.I / 16, slots);
  if (gu.bK == 128) hipLaunchKernelGGL(moe_gate_up_kernel<128>, g1, dim3(kGuWaves * 64), 0, stream, a);
  else hipLaunchKernelGGL(moe_gate_up_kernel<64>, g1, dim3(kGuWaves * 64), 0, stream, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if ((e = launch_quant_act(ws.h, P, s.I, ws.qh, ws.sh, stream)) != hipSuccess) return e;
  const dim3 g2(s.H / 64, slots);
  if (dn.bK == 128) hipLaunchKernelGGL((moe_down_kernel<128, 2>), g2, dim3(512), 0, stream, a);
  else hipLaunchKernelGGL((moe_down_kernel<64, 2>), g2, dim3(512), 0, stream, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(moe_combine_kernel, dim3((s.H / 4 + 255) / 256, s.M), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace aq
