// Low-rank adapters of many requests at once beside a shared projection:
//   Y[m,n] = Yin[m,n] + scale[a] sum_{r < rank[a]} B[a][n,r] sum_k A[a][r,k] X[m,k],
// a = ids[m]; a token whose id is outside 0 .. L-1 has no adapter.
//
// `shrink` forms v = A x as KS partial sums over column ranges, `expand` adds
// scale B v to the projection's output; all products and sums in FP32 (the
// adapters' BF16 or FP16 values are exact there).  A token is one row or
// column of the products, so neither the order of the tokens nor the mix of
// adapters, nor another request's values, enters its result.  Many tokens are
// first grouped by adapter, by a launch of its own.
//
// Bound: memory.  Few tokens, or tokens with an adapter each, stream their
// adapters, one wave per token and range; many tokens stream X, then Yin and Y
// (a rank-16 adapter does 8 multiply-adds per byte of them) and multiply on the
// matrix cores: adapters in FP32 on the FP32 instructions (154 TFLOP/s), 16-bit
// ones on the BF16 instructions, with FP32 values in three exact pieces.

#include <hip/hip_fp16.h>

#include <type_traits>

#include "aq_device.h"
#include "aq_lds_pipe.h"
#include "aq_quant.h"
#include "aq_routed.h"
#include "aq_tile_stream.h"

namespace aq {
namespace {

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
// 16-bit adapters meet FP32 values on the BF16 matrix instructions, which are 16
// times as fast as the FP32 ones: an FP32 value is the sum of three BF16 ones
// exactly (8 bits of its 24 each, cut off, not rounded; below 2^-102 the last
// pieces fall out of the normal range, by less than 2^-126), an FP16 value of two,
// and a product of two BF16 values is exact in FP32.  Adapters in FP32 take the
// FP32 instructions.
//   The pieces of an infinity are the infinity and NaN, and an infinity on one
// side meets pieces of 0 on the other, so a sum of pieces that is NaN need not be
// one of the values.  Both kernels form these sums anew, from the values: 8192 x
// 4096, rank 16: 99 us with and without the check where nothing is infinite, 105 with
// NaN in 30% of the rows, 194 with an infinity in 1% of them.
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint32_t upper_halves(float lo, float hi) {
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302);
}
__device__ __forceinline__ float below(float x) { return x - __uint_as_float(__float_as_uint(x) & 0xFFFF0000u); }
// The first piece of N values, packed in pairs; what is left replaces them (INF: 0
// of an infinity, whose pieces then add up to it).
template <bool INF = false, int N>
__device__ __forceinline__ void take_piece(float (&x)[N], uint32_t (&o)[N / 2]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    o[i / 2] = upper_halves(x[i], x[i + 1]);
    x[i] = INF && fabsf(x[i]) == INFINITY ? 0.f : below(x[i]);
    x[i + 1] = INF && fabsf(x[i + 1]) == INFINITY ? 0.f : below(x[i + 1]);
  }
}
__device__ __forceinline__ v8bf as_v8bf(const uint32_t (&w)[4]) {
  return __builtin_bit_cast(v8bf, v4u{w[0], w[1], w[2], w[3]});
}
// 8 adapter values as PIECES operands of a BF16 matrix instruction.
template <typename T> constexpr int kPieces = sizeof(T) == 4 ? 0 : 1;
template <> constexpr int kPieces<__half> = 2;
__device__ __forceinline__ void pieces_of(const bf16_t *, const uint32_t (&w)[4], v8bf (&o)[1]) { o[0] = as_v8bf(w); }
__device__ __forceinline__ void pieces_of(const __half *, const uint32_t (&w)[4], v8bf (&o)[2]) {
  float f[8];
  uint32_t p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = *reinterpret_cast<const __half2 *>(&w[i]);
    f[2 * i] = __low2float(h);
    f[2 * i + 1] = __high2float(h);
  }
  take_piece(f, p);
  o[0] = as_v8bf(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = upper_halves(f[2 * i], f[2 * i + 1]);
  o[1] = as_v8bf(p);
}

__device__ __forceinline__ float load1f(const bf16_t *p) { return __uint_as_float((uint32_t)p->bits << 16); }
__device__ __forceinline__ float load1f(const __half *p) { return __half2float(*p); }
__device__ __forceinline__ void load4f(const float *p, float (&o)[4]) {
  const float4 a = *reinterpret_cast<const float4 *>(p);
  o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
}
__device__ __forceinline__ int adapter_of(const LoraArgs &a, int m) {
  const int id = m < a.M ? a.ids[m] : -1;
  return (unsigned)id < (unsigned)a.L ? id : -1;
}
__device__ __forceinline__ int rank_of(const LoraArgs &a, int ad) {
  return a.rank ? min(max(a.rank[ad], 0), a.R) : a.R;
}

// Sums 8 values over the 64 lanes: at distances 1, 2 and 4 a lane hands half
// of its values over and keeps the other half, then its one value is summed at
// 8, 16 and 32 (10 exchanges in place of 48).  Lane l returns the total of
// value 4 (l & 1) + 2 (l >> 1 & 1) + (l >> 2 & 1).
template <int PAT>
__device__ __forceinline__ float swz(float v) {
  return __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), PAT));
}
__device__ __forceinline__ float sum8(const float (&s)[8], int lane) {
  float t[4], u[2];
  const bool b0 = lane & 1, b1 = lane & 2, b2 = lane & 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    t[i] = (b0 ? s[i + 4] : s[i]) +
           __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(b0 ? s[i] : s[i + 4]), 0xB1, 0xF, 0xF, false));
#pragma unroll
  for (int i = 0; i < 2; ++i)
    u[i] = (b1 ? t[i + 2] : t[i]) +
           __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(b1 ? t[i] : t[i + 2]), 0x4E, 0xF, 0xF, false));
  float v = (b2 ? u[1] : u[0]) + swz<0x101F>(b2 ? u[0] : u[1]);
  v += swz<0x201F>(v);
  v += swz<0x401F>(v);
  return v + __shfl_xor(v, 32);
}

// v of one token over columns 64 b0 .. 64 b1 - 1 by one wave: lane l takes 8
// columns of every 512, a row of A is one coalesced load.  Of the groups of 8
// ranks it takes every gridDim.z-th from blockIdx.z on.
template <typename T>
__device__ __forceinline__ void shrink_token(const LoraArgs &a, int m, int id, int b0, int b1, int lane, float *v) {
  const int rank = __builtin_amdgcn_readfirstlane(rank_of(a, id));
  const T *A = static_cast<const T *>(a.A) + (size_t)id * a.R * a.K;
  const float *x = a.X + (size_t)m * a.K;
  for (int j0 = 8 * blockIdx.z; j0 < rank; j0 += 8 * gridDim.z) {
    float s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = 0.f;
    for (int k = b0 * 64 + 8 * lane; k < b1 * 64; k += 512) {
      float xv[8], w[8][8];
      load8f(x + k, xv);
#pragma unroll
      for (int j = 0; j < 8; ++j) load8f(A + (size_t)min(j0 + j, rank - 1) * a.K + k, w[j]);
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int t = 0; t < 8; ++t) s[j] = fmaf(w[j][t], xv[t], s[j]);
    }
    const float sum = sum8(s, lane);
    const int j = j0 + 4 * (lane & 1) + 2 * (lane >> 1 & 1) + (lane >> 2 & 1);
    if (lane < 8 && j < rank) v[j] = sum;
  }
}

// Few tokens: one wave per token and column range.
template <typename T>
__global__ __launch_bounds__(256) void lora_shrink_rows_kernel(const LoraArgs a) {
  const int lane = threadIdx.x & 63;
  const int m = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int id = __builtin_amdgcn_readfirstlane(adapter_of(a, m));
  if (id < 0) return;
  const int nb = a.K >> 6, ks = blockIdx.y;
  shrink_token<T>(a, m, id, (int)((long long)nb * ks / a.KS), (int)((long long)nb * (ks + 1) / a.KS), lane,
                  a.v + ((size_t)ks * a.M + m) * a.R);
}

// 4 sums over columns k0 .. k1-1 of x with n <= 4 rows of A by one lane, for what the
// pieces made NaN of; given up where all are NaN.
template <typename T>
__device__ __forceinline__ void sum_of_nan(const T *A, const float *x, int K, int k0, int k1, int n, float (&q)[4]) {
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int k = k0; k < k1; k += 8) {
    float xv[8];
    load8f(x + k, xv);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      float w[8], t = i == 0 ? s[0] : i == 1 ? s[1] : i == 2 ? s[2] : s[3];
      load8f(A + (size_t)i * K + k, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) t = fmaf(w[j], xv[j], t);
      s[0] = i == 0 ? t : s[0];
      s[1] = i == 1 ? t : s[1];
      s[2] = i == 2 ? t : s[2];
      s[3] = i == 3 ? t : s[3];
    }
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) any |= i < n && s[i] == s[i];
    if (!any) break;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = i < n ? s[i] : q[i];
}

// ---- many tokens: tiles of up to 64 tokens of one adapter.
//
// One workgroup groups the tokens by adapter (the tokens without one as a last
// group) and cuts every group into tiles {adapter, start, count} over the
// permuted tokens.  A wave adds its tokens of one adapter with one LDS atomic.
// The order inside a group depends on the order of these, a token's result
// does not: it is a row or column of its own in every product.
struct LoraTile {
  int32_t ad, start, count, pad;
};
__device__ __forceinline__ int32_t *perm_of(const LoraArgs &a) { return a.lists + 4; }
__device__ __forceinline__ LoraTile *tiles_of(const LoraArgs &a) {
  return reinterpret_cast<LoraTile *>(a.lists + 4 + ((a.M + 3) & ~3));
}
// Tile t; false past the last.  Its fields are read along with the number of
// tiles, not after it (the places past the last hold anything).
__device__ __forceinline__ bool tile_at(const LoraArgs &a, int t, int &ad, int &cnt, const int32_t *&rows) {
  const LoraTile *tl = tiles_of(a) + t;
  const int n = uload(a.lists), start = uload(&tl->start);
  ad = uload(&tl->ad);
  cnt = uload(&tl->count);
  asm volatile("" ::"s"(n), "s"(start), "s"(ad), "s"(cnt));
  rows = perm_of(a) + start;
  return t < n;
}
constexpr int kListsU = 8;  // tokens per thread that stay in registers
template <bool ONE>
__global__ __launch_bounds__(1024) void lora_lists_kernel(const LoraArgs a) {
  extern __shared__ int32_t grp_lds[];
  __shared__ int wtok[16], wtile[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int G = a.L + 1;
  // per group: tokens, first tile, first place (of one group more)
  int32_t *cnt = grp_lds, *tile0 = cnt + G, *start = tile0 + G;
  for (int i = tid; i < G; i += 1024) cnt[i] = 0;
  __syncthreads();
  // Places of the tokens m0 + 1024 u + (lane of the wave) in their groups
  auto places = [&](int m0, int (&grp)[kListsU], int (&pos)[kListsU]) __attribute__((always_inline)) {
    int id[kListsU];
#pragma unroll
    for (int u = 0; u < kListsU; ++u) id[u] = a.ids[min(m0 + 1024 * u + tid, a.M - 1)];
    // all loads before the first use (the compiler makes each one conditional on
    // its use and waits for them one by one: 9.5 us for 8192 tokens)
    asm volatile("" : "+v"(id[0]), "+v"(id[1]), "+v"(id[2]), "+v"(id[3]), "+v"(id[4]), "+v"(id[5]), "+v"(id[6]), "+v"(id[7]));
    static_assert(kListsU == 8, "");
#pragma unroll
    for (int u = 0; u < kListsU; ++u)
      grp[u] = m0 + 1024 * u + tid >= a.M ? -1 : (unsigned)id[u] < (unsigned)a.L ? id[u] : a.L;
#pragma unroll
    for (int u = 0; u < kListsU; ++u) {
      // one LDS atomic per wave where its tokens share an adapter, else one per
      // token; none waits for another
      const int at = __builtin_amdgcn_readfirstlane(grp[u]);
      pos[u] = 0;
      if (__ballot(grp[u] != at) == 0) {
        if (at >= 0 && lane == 0) pos[u] = atomicAdd(&cnt[at], 64);
      } else if (grp[u] >= 0) {
        pos[u] = atomicAdd(&cnt[grp[u]], 1);
      }
    }
#pragma unroll
    for (int u = 0; u < kListsU; ++u) {
      const int at = __builtin_amdgcn_readfirstlane(grp[u]);
      if (__ballot(grp[u] != at) == 0) pos[u] = __builtin_amdgcn_readfirstlane(pos[u]) + lane;
    }
  };
  int grp[kListsU], pos[kListsU];
  for (int m0 = 0; m0 < a.M; m0 += 1024 * kListsU) places(m0, grp, pos);  // (ONE: once)
  __syncthreads();
  // exclusive scans over the groups: tokens before, tiles before (a thread
  // takes consecutive groups)
  const int per = (G + 1023) / 1024, g0 = min(tid * per, G), g1 = min(g0 + per, G);
  int tok = 0, til = 0;
  for (int i = g0; i < g1; ++i) {
    tok += cnt[i];
    til += (cnt[i] + 63) >> 6;
  }
  int s = tok, t = til;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int ps = __shfl_up(s, o), pt = __shfl_up(t, o);
    if (lane >= o) {
      s += ps;
      t += pt;
    }
  }
  if (lane == 63) {
    wtok[wave] = s;
    wtile[wave] = t;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 15; ++w) {
    s += w < wave ? wtok[w] : 0;
    t += w < wave ? wtile[w] : 0;
  }
  if (tid == 1023) {
    a.lists[0] = t;
    start[G] = s;
  }
  s -= tok;
  t -= til;
  for (int i = g0; i < g1; ++i) {
    start[i] = s;
    tile0[i] = t;
    s += cnt[i];
    t += (cnt[i] + 63) >> 6;
  }
  __syncthreads();
  LoraTile *tiles = tiles_of(a);
  int32_t *perm = perm_of(a);
  // a token goes to its place; the first of every 64 places writes the tile
  auto write = [&](int m0) __attribute__((always_inline)) {
    int at[kListsU], end[kListsU], tile[kListsU];
#pragma unroll
    for (int u = 0; u < kListsU; ++u) {
      const int g = max(grp[u], 0);
      at[u] = start[g] + pos[u];
      end[u] = start[g + 1];
      tile[u] = tile0[g] + (pos[u] >> 6);
    }
#pragma unroll
    for (int u = 0; u < kListsU; ++u) {
      const int g = grp[u];
      if (g < 0) continue;
      perm[at[u]] = m0 + 1024 * u + tid;
      if ((pos[u] & 63) == 0) tiles[tile[u]] = LoraTile{g < a.L ? g : -1, at[u], min(64, end[u] - at[u]), 0};
    }
  };
  if constexpr (ONE) {
    write(0);
  } else {
    for (int i = tid; i < G; i += 1024) cnt[i] = 0;
    __syncthreads();
    for (int m0 = 0; m0 < a.M; m0 += 1024 * kListsU) {
      places(m0, grp, pos);
      write(m0);
    }
  }
}

// A 1 KB piece of a tile: 64 lanes x 16 bytes from the lanes' addresses to
// consecutive LDS bytes.
typedef const __attribute__((address_space(1))) void *global_ptr_t;
__device__ __forceinline__ void piece(const void *p, void *lds) {
  __builtin_amdgcn_global_load_lds((global_ptr_t)p, (lds_ptr_t)lds, 16, 0, 0);
}

// shrink: one workgroup of 8 waves per tile and column range, 16 tokens for
// every two waves, which take half of a step's columns each.  The ranges of
// one tile are neighbours in the grid, so that what runs at one time covers
// whole rows (reading X alone: 23 us for 8192 x 4096 against 28 us with the
// tiles as neighbours).  X and A go through LDS in steps of 64 columns, three
// steps deep (operands read as aq_lds_pipe.h says: 8192 x 4096: 34 us against
// 38 us; 2048 x 5120, rank 64 in FP32: 18.5 against 24.5), by loads whose lanes
// read whole 128-byte lines; 16-byte granule
// q of row r sits at place q ^ r (r modulo the granules of a row), so that the
// 16 rows of an operand read fall in different banks.  RT: 16-rank tiles.
template <typename T, int RT>
__global__ __launch_bounds__(512) void lora_shrink_kernel(const LoraArgs a) {
  constexpr int XB = 64 * 256, AROW = 64 * sizeof(T);
  constexpr int AB = 16 * RT * AROW < 8192 ? 8192 : 16 * RT * AROW;  // one piece per wave at least
  constexpr int AG = AROW / 16, AP = AB / 8192, PIECES = 2 + AP;
  extern __shared__ __align__(16) uint8_t lds[];  // [ST][XB + AB]
  const int tile = (int)(blockIdx.x / (unsigned)a.KS), ks = (int)(blockIdx.x % (unsigned)a.KS);
  int ad, cnt;
  const int32_t *rows;
  if (!tile_at(a, tile, ad, cnt, rows) || ad < 0) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, i16 = lane & 15, tw = wave >> 1, half = wave & 1;
  const int nb = a.K >> 6;
  const int b0 = (int)((long long)nb * ks / a.KS), b1 = (int)((long long)nb * (ks + 1) / a.KS);
  const char *xp[2], *ap[AP];
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // 4 rows of 16 granules a piece; rows past the end read the last
    const int r = (2 * wave + i) * 4 + (lane >> 4);
    xp[i] = reinterpret_cast<const char *>(a.X + (size_t)rows[min(r, cnt - 1)] * a.K) + 16 * ((lane & 15) ^ (r & 15));
  }
#pragma unroll
  for (int i = 0; i < AP; ++i) {
    const int r = (AP * wave + i) * (64 / AG) + lane / AG;
    ap[i] = reinterpret_cast<const char *>(static_cast<const T *>(a.A) + ((size_t)ad * a.R + min(r, a.R - 1)) * a.K) +
            16 * ((lane % AG) ^ (r & (AG - 1)));
  }
  // A wave whose 8 rows of X hold no token leaves them as they are: a token is a
  // column of the products, so what they hold reaches no other's.
  const bool xlive = 8 * wave < cnt;
  auto fetch = [&](int b, int at) __attribute__((always_inline)) {
    b = min(b, b1 - 1);  // past the range: the last step again (never multiplied)
    uint8_t *to = lds + at * (XB + AB);
    if (xlive) {
#pragma unroll
      for (int i = 0; i < 2; ++i) piece(xp[i] + (size_t)b * 256, to + (2 * wave + i) * 1024);
    }
#pragma unroll
    for (int i = 0; i < AP; ++i) piece(ap[i] + (size_t)b * AROW, to + XB + (AP * wave + i) * 1024);
  };
  constexpr int RB = RT < 4 ? RT : 4;  // rank tiles a read
  // the lane's pieces of a step in stage 0 (rank tile 0), the wave's 32 columns:
  // FP32: 4 columns of every 16; 16-bit: 8 columns together
  uint32_t xa[2], aa[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int q = sizeof(T) == 4 ? 4 * (2 * half + p) + g : 8 * half + 2 * g + p;
    xa[p] = lds_address(lds) + (16 * tw + i16) * 256 + 16 * (q ^ i16);
    aa[p] = lds_address(lds) + XB + i16 * AROW + 16 * (sizeof(T) == 4 ? q ^ i16 : (4 * half + g) ^ (i16 & 7));
  }
  const bool live = 16 * tw < cnt;  // any token for the wave
  v4f acc[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = v4f{0.f, 0.f, 0.f, 0.f};
  fetch(b0, 0);
  fetch(b0 + 1, 1);
  int at = 0;
  for (int b = b0; b < b1; ++b) {
    // this step's pieces have landed (the next one's may be open), for every wave
    if (xlive) __builtin_amdgcn_s_waitcnt(0x0070 | PIECES);  // vmcnt(PIECES), lgkmcnt(0)
    else __builtin_amdgcn_s_waitcnt(0x0070 | (PIECES - 2));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    // the place of the step before last: every wave has multiplied it
    fetch(b + 2, at >= 1 ? at - 1 : 2);
    if (live) {
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint32_t xs = xa[p] + at * (XB + AB), as = aa[p] + at * (XB + AB);
#pragma unroll
          for (int r = 0; r < RT; r += RB) {
            uint32_t ws[RB];
            v4f x, w[RB];
#pragma unroll
            for (int i = 0; i < RB; ++i) ws[i] = as + (r + i) * 16 * AROW;
            lds_read(xs, ws, x, w);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
              for (int i = 0; i < RB; ++i)
                acc[r + i] = __builtin_amdgcn_mfma_f32_16x16x4f32(w[i][t], x[t], acc[r + i], 0, 0, 0);
          }
        }
      } else {
        const uint32_t xs[2] = {xa[0] + at * (XB + AB), xa[1] + at * (XB + AB)}, as = aa[0] + at * (XB + AB);
        v8bf xp[3];
#pragma unroll
        for (int r = 0; r < RT; r += RB) {
          uint32_t ws[RB];
          v4f xv[2], w[RB];
#pragma unroll
          for (int i = 0; i < RB; ++i) ws[i] = as + (r + i) * 16 * AROW;
          lds_read(xs, ws, xv, w);
          if (r == 0) {
            float f[8];
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = xv[i >> 2][i & 3];
#pragma unroll
            for (int i = 0; i < 3; ++i) {
              take_piece(f, o);
              xp[i] = as_v8bf(o);
            }
          }
#pragma unroll
          for (int i = 0; i < RB; ++i) {
            const uint32_t raw[4] = {__float_as_uint(w[i][0]), __float_as_uint(w[i][1]), __float_as_uint(w[i][2]),
                                     __float_as_uint(w[i][3])};
            v8bf wp[kPieces<T>];
            pieces_of(static_cast<const T *>(nullptr), raw, wp);
#pragma unroll
            for (int k = 2; k >= 0; --k)
#pragma unroll
              for (int m = kPieces<T> - 1; m >= 0; --m)
                acc[r + i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wp[m], xp[k], acc[r + i], 0, 0, 0);
          }
        }
      }
    }
    at = at == 2 ? 0 : at + 1;
  }
  // every load into LDS and every read of it is done; the halves meet there
  __builtin_amdgcn_s_waitcnt(0x0070);
  __syncthreads();
  float4 *red = reinterpret_cast<float4 *>(lds) + (size_t)tw * RT * 64 + lane;
  if (half) {
#pragma unroll
    for (int r = 0; r < RT; ++r) red[r * 64] = make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
  }
  __syncthreads();
  if (half || 16 * tw + i16 >= cnt) return;
  // lane: ranks 16r + 4g .. + 3 of token i16 (what lies beyond the adapter's
  // rank is not read)
  const size_t tok = rows[16 * tw + i16];
  float *v = a.v + ((size_t)ks * a.M + tok) * a.R;
  const int rank = sizeof(T) == 2 ? rank_of(a, ad) : 0;
#pragma unroll
  for (int r = 0; r < RT; ++r)
    if (16 * r + 4 * g < a.R) {
      const float4 o = red[r * 64];
      float q[4] = {acc[r][0] + o.x, acc[r][1] + o.y, acc[r][2] + o.z, acc[r][3] + o.w};
      if constexpr (sizeof(T) == 2) {
        const float all = (q[0] + q[1]) + (q[2] + q[3]);
        const int r0 = 16 * r + 4 * g, n = min(4, rank - r0);
        if (all != all && n > 0)
          sum_of_nan(static_cast<const T *>(a.A) + ((size_t)ad * a.R + r0) * a.K, a.X + tok * a.K, a.K, 64 * b0, 64 * b1,
                     n, q);
      }
      *reinterpret_cast<float4 *>(v + 16 * r + 4 * g) = make_float4(q[0], q[1], q[2], q[3]);
    }
}

// 8 values of v at ranks k .. of token m, the partial sums added in increasing
// order, times the adapter's scale; 0 beyond its rank.
__device__ __forceinline__ void load_v(const LoraArgs &a, int m, int k, int rank, float scale, float (&v)[8]) {
#pragma unroll
  for (int t = 0; t < 8; ++t) v[t] = 0.f;
  if (k >= rank) return;
#pragma unroll 4
  for (int s = 0; s < a.KS; ++s) {
    float q[8];
    load8f(a.v + ((size_t)s * a.M + m) * a.R + k, q);
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] += q[t];
  }
#pragma unroll
  for (int t = 0; t < 8; ++t) v[t] = k + t < rank ? v[t] * scale : 0.f;
}

// 8 adapter values (4 in FP32) as they are stored, widened when they are used.
template <typename T> struct Raw8 {
  uint4 v;
  __device__ __forceinline__ void load(const T *p) { v = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void widen(float (&o)[8]) const { load8f(reinterpret_cast<const T *>(&v), o); }
};
template <> struct Raw8<float> {
  float4 v[2];
  __device__ __forceinline__ void load(const float *p) {
    v[0] = reinterpret_cast<const float4 *>(p)[0];
    v[1] = reinterpret_cast<const float4 *>(p)[1];
  }
  __device__ __forceinline__ void widen(float (&o)[8]) const { load8f(reinterpret_cast<const float *>(v), o); }
};
struct Raw4 {
  float4 v;
  __device__ __forceinline__ void load(const float *p) { v = *reinterpret_cast<const float4 *>(p); }
  __device__ __forceinline__ void widen(float (&o)[4]) const { o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w; }
};

// Few tokens: LPR lanes per row of B, 8 ranks each; a wave takes 64 / LPR rows
// a load, UR loads at once and NCH such chunks one after another, the next
// one's loads in flight while one is multiplied.
template <typename T, int LPR>
__global__ __launch_bounds__(256) void lora_expand_rows_kernel(const LoraArgs a, int NCH) {
  constexpr int RPL = 64 / LPR, UR = sizeof(T) == 4 ? 4 : 8, ROWS = RPL * UR;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = blockIdx.y;
  const int id = __builtin_amdgcn_readfirstlane(adapter_of(a, m));
  const int n0 = (blockIdx.x * 4 + wave) * ROWS * NCH, n1 = min(n0 + ROWS * NCH, a.N);
  const float *yi = a.Yin + (size_t)m * a.ldyin;
  float *yo = a.Y + (size_t)m * a.ldy;
  if (id < 0) {
    if (a.Yin != a.Y)
      for (int n = n0 + lane; n < n1; n += 64) yo[n] = yi[n];
    return;
  }
  if (n0 >= n1) return;
  const int sub = lane % LPR, row = lane / LPR, k = 8 * sub;
  const int rank = __builtin_amdgcn_readfirstlane(rank_of(a, id));
  const T *B = static_cast<const T *>(a.B) + (size_t)id * a.N * a.R + k;
  struct Chunk {
    Raw8<T> w[UR];
    float y[(UR + LPR - 1) / LPR];
  } ch[2];
  // (lanes beyond the rank load nothing: 8 tokens of FP32 adapters, rank up to
  // 128: 11.6 us, loading all 14.4; chunks past the end load the last row)
  auto fetch = [&](int n, Chunk &c) __attribute__((always_inline)) {
    if (k < rank) {
#pragma unroll
      for (int u = 0; u < UR; ++u) c.w[u].load(B + (size_t)min(n + u * RPL + row, a.N - 1) * a.R);
    }
    // after the sums lane sub stores loads sub, sub + LPR, ..
#pragma unroll
    for (int u0 = 0; u0 < UR; u0 += LPR) c.y[u0 / LPR] = yi[min(n + (u0 + sub) * RPL + row, a.N - 1)];
  };
  fetch(n0, ch[0]);
  float v[8];
  load_v(a, m, k, rank, a.scale ? a.scale[id] : 1.f, v);
  auto compute = [&](int n, Chunk &c) __attribute__((always_inline)) {
    float s[UR];
#pragma unroll
    for (int u = 0; u < UR; ++u) {
      float w[8];
      s[u] = 0.f;
      c.w[u].widen(w);
#pragma unroll
      for (int t = 0; t < 8; ++t) s[u] = fmaf(k + t < rank ? w[t] : 0.f, v[t], s[u]);
    }
#pragma unroll
    for (int u = 0; u < UR; ++u) {
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) s[u] += __shfl_xor(s[u], o);
    }
#pragma unroll
    for (int u0 = 0; u0 < UR; u0 += LPR) {
      float y = s[u0];
#pragma unroll
      for (int u = 1; u < LPR; ++u)
        if (u0 + u < UR) y = sub == u ? s[u0 + u] : y;
      const int at = n + (u0 + sub) * RPL + row;
      if (u0 + sub < UR && at < n1) yo[at] = c.y[u0 / LPR] + y;
    }
  };
#pragma unroll 1
  for (int n = n0; n < n1; n += 2 * ROWS) {
    fetch(n + ROWS, ch[1]);
    compute(n, ch[0]);
    fetch(n + 2 * ROWS, ch[0]);
    if (n + ROWS < n1) compute(n + ROWS, ch[1]);
  }
}

// expand: one workgroup of 4 waves per tile, a wave per NB blocks of 32
// features on 32 x 32 matrix instructions (the tokens as rows); a block of B serves
// both halves of the tile, and the next block's B and the next half's Yin are
// in flight while one is multiplied.  (Whole tiles of Yin held ahead took 64
// registers and a wave per SIMD: 2048 x 7168, rank 64: 46 us against 42.)  The column groups of one tile are neighbours in the
// grid, so that what runs at one time covers whole rows.  v is added up and
// scaled once per workgroup, in LDS.  The products pass through the wave's own LDS so that Yin and Y are read and
// written 16 bytes a lane, whole 128-byte lines of 8 rows at a time (4 bytes a
// lane, two rows: 77 us against 64 us for 8192 x 4096; with the column groups
// as neighbours 58 us, where a copy of Y takes 52 us).  RQ: 8-rank steps.
typedef float v16f __attribute__((ext_vector_type(16)));
// Waves per SIMD that the registers of RQ steps leave room for.
constexpr int expand_waves(int RQ, int bytes) { return RQ <= 2 ? 4 : RQ == 4 ? (bytes == 2 ? 4 : 3) : RQ == 8 ? (bytes == 2 ? 3 : 2) : 1; }
template <typename T, int RQ>
__global__ __launch_bounds__(256, expand_waves(RQ, sizeof(T))) void lora_expand_kernel(const LoraArgs a, int NB) {
  constexpr bool F32 = sizeof(T) == 4;
  // a lane's ranks of a row of B: UN units of U (which rank meets which product
  // of the FP32 instruction is free, as long as v agrees)
  constexpr int U = F32 && RQ == 1 ? 4 : 8, UN = RQ == 1 ? 1 : RQ / 2;
  typedef std::conditional_t<U == 4, Raw4, Raw8<T>> Raw;
  // v in LDS: FP32, or three pieces; rows 16 bytes apart in the banks
  constexpr int VS = F32 ? 8 * RQ + 4 : 8 * UN + 4;  // row stride, words
  constexpr int OS = 36;
  __shared__ __align__(16) float vs[(F32 ? 1 : 3) * 64 * VS];
  __shared__ __align__(16) float os[4][32 * OS];
  int ad, cnt;
  const int32_t *rows;
  if (!tile_at(a, blockIdx.y, ad, cnt, rows) || (ad < 0 && a.Yin == a.Y)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, i32 = lane & 31;
  const int rank_ = ad >= 0 ? min(max(a.rank ? uload(a.rank + ad) : a.R, 0), a.R) : 0, ldy_ = (int)a.ldy;
  const int nb0 = blockIdx.x * 4 * NB + wave, nb1 = min((int)(blockIdx.x + 1) * 4 * NB, a.N >> 5);
  // the lane's 8 rows of Yin and Y (8 j + lane / 8; rows past the end read the
  // last and are not written), at column 4 (lane % 8)
  uint32_t m[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) m[j] = rows[min(8 * j + (lane >> 3), cnt - 1)];
  const float *yin = a.Yin + 4 * (lane & 7);
  float *yout = a.Y + 4 * (lane & 7);
  const T *Bp = static_cast<const T *>(a.B) + (size_t)max(ad, 0) * a.N * a.R;
  // B double-buffered, Yin by halves of the tile: y[c] holds tokens 32c ..
  Raw w[2][UN];  // row n of B: ranks U (2q + h) ..
  float4 y[2][4];
  const bool two = cnt > 32;
  auto fetch_w = [&](int nb, Raw (&o)[UN]) __attribute__((always_inline)) {
    nb = min(nb, (a.N >> 5) - 1);  // past the end: any block (not used)
    const T *B = Bp + (size_t)(nb * 32 + i32) * a.R;
#pragma unroll
    for (int q = 0; q < UN; ++q) o[q].load(B + min(U * (2 * q + h), a.R - U));
  };
  auto fetch_y = [&](int nb, int c) __attribute__((always_inline)) {
    nb = min(nb, (a.N >> 5) - 1);
    int ldyin = (int)a.ldyin;  // (at most 2^22)
    asm volatile("" : "+s"(ldyin));
#pragma unroll
    for (int j = 0; j < 4; ++j)
      y[c][j] = *reinterpret_cast<const float4 *>(yin + (uint64_t)m[4 * c + j] * (uint32_t)ldyin + nb * 32);
  };
  fetch_w(nb0, w[0]);
  fetch_y(nb0, 0);
  {
    // thread: ranks 4 (thread % 4) + 16 c .. of token thread / 4, the partial
    // sums of all its ranks loaded side by side and added in increasing order
    constexpr int NC = (RQ + 1) / 2;
    const int t = threadIdx.x >> 2, k0 = 4 * (threadIdx.x & 3);
    const size_t tok = rows[min(t, cnt - 1)];
    const float scale = ad >= 0 && a.scale ? uload(a.scale + ad) : 1.f;
    float v[NC][4];
#pragma unroll
    for (int c = 0; c < NC; ++c) v[c][0] = v[c][1] = v[c][2] = v[c][3] = 0.f;
#pragma unroll(RQ < 8 ? 4 : 2)
    for (int s = 0; s < a.KS; ++s) {
      const float *p = a.v + ((size_t)s * a.M + tok) * a.R + k0;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float q[4] = {0.f, 0.f, 0.f, 0.f};
        if (t < cnt && k0 + 16 * c < rank_) load4f(p + 16 * c, q);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[c][i] += q[i];
      }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int k = k0 + 16 * c;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[c][i] = k + i < rank_ ? v[c][i] * scale : 0.f;
      if constexpr (F32) {
        if (k < 8 * RQ) *reinterpret_cast<float4 *>(vs + t * VS + k) = make_float4(v[c][0], v[c][1], v[c][2], v[c][3]);
      } else {
        // (k < 16 UN; 0 beyond the rank)
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          uint32_t o[2];
          take_piece<true>(v[c], o);
          *reinterpret_cast<uint2 *>(vs + (64 * i + t) * VS + k / 2) = make_uint2(o[0], o[1]);
        }
      }
    }
  }
  __syncthreads();
  float *o = os[wave];
  // The lane's sums of a block that the pieces made NaN of, from v and B themselves;
  // a token whose own v is NaN costs a read of LDS.
  auto nan_anew = [&](int nb, int c) __attribute__((always_inline)) {
    if constexpr (!F32) {
      const T *B = Bp + (size_t)(nb * 32 + i32) * a.R;
      const uint16_t *vp = reinterpret_cast<const uint16_t *>(vs);
#pragma unroll 1
      for (int i = 0; i < 16; ++i) {
        const int t = 8 * (i >> 2) + 4 * h + (i & 3);
        float s = o[t * OS + i32];
        if (32 * c + t >= cnt || s == s) continue;
        s = 0.f;
#pragma unroll 1
        for (int k = 0; k < rank_ && s == s; ++k) {
          float v = 0.f;
#pragma unroll
          for (int p = 0; p < 3; ++p) v += __uint_as_float((uint32_t)vp[2 * (64 * p + 32 * c + t) * VS + k] << 16);
          s = v == v ? fmaf(load1f(B + k), v, s) : v;
        }
        o[t * OS + i32] = s;
      }
    }
  };
  auto compute = [&](int nb, int c, const Raw (&wr)[UN]) __attribute__((always_inline)) {
    v16f acc = {};
    // v, the masks and the rows' addresses are formed anew, not kept in registers
    // from block to block
    int rank = rank_, ldy = ldy_;
    asm volatile("" : "+s"(rank), "+s"(ldy)::"memory");
#pragma unroll
    for (int q = 0; q < UN; ++q) {
      const int k = U * (2 * q + h);
      if constexpr (F32) {
        float v[U], w[U];
        wr[q].widen(w);
#pragma unroll
        for (int i = 0; i < U; ++i) w[i] = k + i < rank ? w[i] : 0.f;  // nothing beyond the adapter's rank enters
#pragma unroll
        for (int i = 0; i < U; i += 4) {
          const float4 p = *reinterpret_cast<const float4 *>(vs + (32 * c + i32) * VS + k + i);
          v[i] = p.x; v[i + 1] = p.y; v[i + 2] = p.z; v[i + 3] = p.w;
        }
#pragma unroll
        for (int i = 0; i < U; ++i) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(v[i], w[i], acc, 0, 0, 0);
      } else {
        uint32_t raw[4] = {wr[q].v.x, wr[q].v.y, wr[q].v.z, wr[q].v.w};
        if (16 * q + 16 > rank) {  // nothing beyond the adapter's rank enters
#pragma unroll
          for (int i = 0; i < 4; ++i)
            raw[i] &= (k + 2 * i < rank ? 0xFFFFu : 0u) | (k + 2 * i + 1 < rank ? 0xFFFF0000u : 0u);
        }
        v8bf wp[kPieces<T>];
        pieces_of(static_cast<const T *>(nullptr), raw, wp);
#pragma unroll
        for (int i = 2; i >= 0; --i) {
          const v8bf v = *reinterpret_cast<const v8bf *>(vs + (64 * i + 32 * c + i32) * VS + k / 2);
#pragma unroll
          for (int m = kPieces<T> - 1; m >= 0; --m) acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, wp[m], acc, 0, 0, 0);
        }
      }
    }
    // element i: token 8 (i / 4) + 4h + i % 4 of the half, feature i32
#pragma unroll
    for (int i = 0; i < 16; ++i) o[(8 * (i >> 2) + 4 * h + (i & 3)) * OS + i32] = acc[i];
    if constexpr (!F32) {
      float all = 0.f;
#pragma unroll
      for (int i = 0; i < 16; i += 4) all += (acc[i] + acc[i + 1]) + (acc[i + 2] + acc[i + 3]);
      if (all != all) nan_anew(nb, c);
    }
    // the wave's own LDS: in order, no barrier
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 p = *reinterpret_cast<const float4 *>(o + (8 * j + (lane >> 3)) * OS + 4 * (lane & 7));
      const float4 q = y[c][j];
      if (32 * c + 8 * j + (lane >> 3) < cnt)
        *reinterpret_cast<float4 *>(yout + (uint64_t)m[4 * c + j] * (uint32_t)ldy + nb * 32) =
            ad >= 0 ? make_float4(q.x + p.x, q.y + p.y, q.z + p.z, q.w + p.w) : q;
    }
  };
  auto step = [&](int nb, const Raw (&cur)[UN], Raw (&next)[UN]) __attribute__((always_inline)) {
    if (two) fetch_y(nb, 1);
    fetch_w(nb + 4, next);
    compute(nb, 0, cur);
    fetch_y(nb + 4, 0);
    if (two) compute(nb, 1, cur);
  };
#pragma unroll 1
  for (int nb = nb0; nb < nb1; nb += 8) {
    step(nb, w[0], w[1]);
    if (nb + 4 < nb1) step(nb + 4, w[1], w[0]);
  }
}

template <typename T, int RT>
void launch_shrink(const LoraArgs &a, hipStream_t stream) {
  constexpr int AB = 16 * RT * 64 * (int)sizeof(T) < 8192 ? 8192 : 16 * RT * 64 * (int)sizeof(T);
  constexpr size_t lds = 3 * (64 * 256 + AB);
  if (lds > 64 * 1024)
    (void)hipFuncSetAttribute(reinterpret_cast<const void *>(lora_shrink_kernel<T, RT>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  hipLaunchKernelGGL((lora_shrink_kernel<T, RT>), dim3(lora_max_tiles(a.M, a.L) * a.KS), dim3(512), lds, stream, a);
}
template <typename T, int RQ>
void launch_expand(const LoraArgs &a, hipStream_t stream) {
  // Blocks per wave: 4, or 2 where that would leave less than two workgroups
  // per CU.  (2048 x 7168, rank 64 in FP32: 42 us with 4, 44 with 2, 53 with 8;
  // 6418 x 2816, rank 8: 33, 34 and 35; 8192 x 4096, rank 16: 58, 55 and 70;
  // 463 x 10496, rank 64: 19.9 with 4, 18.0 with 2, 29 with 8.)
  const int tiles = lora_max_tiles(a.M, a.L), nblocks = a.N / 32;
  const int NB = (long long)tiles * ((nblocks + 15) / 16) < 512 ? 2 : 4;
  hipLaunchKernelGGL((lora_expand_kernel<T, RQ>), dim3((nblocks + 4 * NB - 1) / (4 * NB), tiles), dim3(256), 0, stream,
                     a, NB);
}
template <typename T, int LPR>
void launch_expand_rows(const LoraArgs &a, hipStream_t stream) {
  // chunks per wave: as few as leave one round of at most 14 waves per CU (what
  // the registers hold), at most 4 (333 tokens, N 9728, rank 8: 10.5 us with 2,
  // 12.9 with 1 and a second round; with 4, half of the waves, 15.4)
  const int rows = 64 / LPR * (sizeof(T) == 4 ? 4 : 8);
  const long long waves = ((long long)a.M * ((a.N + rows - 1) / rows) + 3583) / 3584;
  const int nch = waves < 1 ? 1 : waves > 4 ? 4 : (int)waves, per = 4 * nch * rows;
  hipLaunchKernelGGL((lora_expand_rows_kernel<T, LPR>), dim3((a.N + per - 1) / per, a.M), dim3(256), 0,
                     stream, a, nch);
}

template <typename T>
hipError_t launch_t(const LoraArgs &a, hipStream_t stream) {
  hipError_t e;
  if (lora_by_rows(a.M, a.L, a.K, a.N, a.R, a.type)) {
    // groups of 8 ranks side by side while the waves fit the chip (16 per CU):
    // one after another each is a load round trip (16 tokens, rank 128: 6 us
    // against 20; 64 tokens, rank 32: 5.6 against 9.4)
    const long long waves = 4LL * ((a.M + 3) / 4) * a.KS, most = 4096 / waves;
    const int Z = (int)(most < 1 ? 1 : most > (a.R + 7) / 8 ? (a.R + 7) / 8 : most);
    hipLaunchKernelGGL(lora_shrink_rows_kernel<T>, dim3((a.M + 3) / 4, a.KS, Z), dim3(256), 0, stream, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (a.R <= 8) launch_expand_rows<T, 1>(a, stream);
    else if (a.R <= 16) launch_expand_rows<T, 2>(a, stream);
    else if (a.R <= 32) launch_expand_rows<T, 4>(a, stream);
    else if (a.R <= 64) launch_expand_rows<T, 8>(a, stream);
    else launch_expand_rows<T, 16>(a, stream);
    return hipGetLastError();
  }
  const size_t lds = 12 * (size_t)(a.L + 1) + 4;
  const auto lists = a.M <= 1024 * kListsU ? lora_lists_kernel<true> : lora_lists_kernel<false>;
  if (lds > 64 * 1024)
    (void)hipFuncSetAttribute(reinterpret_cast<const void *>(lists), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  hipLaunchKernelGGL(lists, dim3(1), dim3(1024), lds, stream, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (a.R <= 16) launch_shrink<T, 1>(a, stream);
  else if (a.R <= 32) launch_shrink<T, 2>(a, stream);
  else if (a.R <= 64) launch_shrink<T, 4>(a, stream);
  else launch_shrink<T, 8>(a, stream);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (sizeof(T) == 4 && a.R <= 8) launch_expand<T, sizeof(T) == 4 ? 1 : 2>(a, stream);
  else if (a.R <= 16) launch_expand<T, 2>(a, stream);
  else if (a.R <= 32) launch_expand<T, 4>(a, stream);
  else if (a.R <= 64) launch_expand<T, 8>(a, stream);
  else launch_expand<T, 16>(a, stream);
  return hipGetLastError();
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
