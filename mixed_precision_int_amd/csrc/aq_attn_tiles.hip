// Attention over the 4-bit cache for prompts: bound by the matrix instructions and the softmax's vector
// instructions, whose times nearly add up.  6000 tokens, 32 heads over 8 of 128, take 594 us (640 to 790 in the first 40 calls
// behind a pause, while the clock settles): 295 GFLOP, 0.50 PFLOP/s,
// each product twice for the two pieces of q or of a weight.  Matrix cores busy 43% of it, the vector ALU 50%, both
// at once 14%; without the widening it takes 70 us less, with half of the products 135, without the
// exponentials 60.  Tried and slower: the next keys' scores formed ahead 587 against 571 at the time, eight waves and
// 128 keys a tile 648, 64 rows to a wave 1187 (one wave to a SIMD, spilled).
//
// A workgroup takes 128 rows of one sequence and key/value head, 32 to each of
// four waves, and walks its keys.  Each tile of keys is widened to FP16 once, by
// all waves, into one of two stages of LDS, keys by feature and values
// transposed (token by token, the widening would cost each wave as much as the
// softmax); the codes of the next tile are on their way meanwhile.
//
// A wave forms S^T = K Q^T with 32 x 32 x 16 products, whose registers are the
// weights' operand of O^T = V^T P^T as they stand (aq_attn_rows.hip): lane % 32
// is the query in all of it, so that maximum, sum and rescaling need one
// exchange between the two halves of the wave.

#include "aq_attn.h"

namespace aq {
namespace {

// q times scale * log2(e) is held times 2^kQ: its two pieces then keep 22 bits for rows whose
// largest value lies within 2^-9 and 2^7, and rows beyond take a power of two of their own.
constexpr int kQ = 8;
constexpr int kWaves = 4, kRows = 32 * kWaves;
static_assert(kRows == kAttnTileRows, "planned on the host");

// A stage of LDS: keys by feature, values transposed.  Rows are 16 bytes longer than what
// they hold, so that 16 neighbouring ones begin in different banks and a chunk's place
// in its row is an immediate offset.  Feature 8f + e of the values is row e * D/8 + f: the
// threads that widen neighbouring eights of features write neighbouring rows.
template <int D>
struct Stage {
  static constexpr int KT = 8192 / D;                    // keys a tile: 64 (D = 128) or 128 (D = 64)
  static constexpr int CK = D / 8 + 1, CV = KT / 8 + 1;  // 16-byte chunks of a key's row, of a feature's row
  h8 k[KT * CK], v[D * CV];
  // of four keys side by side: the key's s times 2^-kQ; of the value's s = f 2^e e, f and 2^-e
  f4 sk[KT / 4], ex[KT / 4], fr[KT / 4], ie[KT / 4];
};

// A thread's share of a tile's codes: 32 features of one key, and 8 features
// of 4 values.
struct Codes {
  u4 k, v, wv;
  uint32_t wk;
};

// A wave's rows into the output, or into the workspace where ranges are joined.
template <int D>
__device__ __forceinline__ void store_rows(const AttnArgs &a, const Rows &r, int item, int head, int ranges,
                                           int wave, int col, int half, const f16v (&o)[D / 32], float M, float l) {
  const int row = r.r0 + 32 * wave + col;
  if (row >= r.rows) return;
  float *out;
  float n = 1.f;
  if (ranges == 1) {
    n = inv_sum(l);
    out = a.out + ((size_t)(r.first + row / a.G) * a.Hq + head * a.G + row % a.G) * D;
  } else {
    out = a.part + (((size_t)item * a.c.heads + head) * kRows + 32 * wave + col) * (D + 4);
    if (half == 0) {
      out[D] = M;
      out[D + 1] = l;
    }
  }
  // row 32 j + 8b + 4 half + i of the product is feature 8f + e with e = row / (D/8),
  // f = row % (D/8)
  constexpr int F = D / 8, B = F / 8;  // D = 128: f from b & 1, e from j and b >> 1; D = 64: f none, e from j and b
#pragma unroll
  for (int bb = 0; bb < B; ++bb)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int at = e * F + 8 * bb;  // the row, but for 4 half + i
        x[e] = o[at / 32][4 * (at % 32 / 8) + i] * n;
      }
      f4 *to = reinterpret_cast<f4 *>(out + 8 * (8 * bb + 4 * half + i));
      to[0] = f4{x[0], x[1], x[2], x[3]};
      to[1] = f4{x[4], x[5], x[6], x[7]};
    }
}

template <int D>
__global__ __launch_bounds__(64 * kWaves, 2) void attn_tiles_kernel(AttnArgs a) {
  using St = Stage<D>;
  constexpr int KT = St::KT, KS = D / 16, DT = D / 32;
  static_assert(KT * D / 32 == 64 * kWaves, "one share per thread");
  extern __shared__ char smem[];
  St *stage = reinterpret_cast<St *>(smem);
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int turn = blockIdx.x / a.c.heads, head = blockIdx.x - turn * a.c.heads;
  const int item = a.items - 1 - turn;  // a sequence's last rows see the most keys: first
  Rows r;
  int split;
  if (!find_rows<kRows, true>(a, item, KT, r, split)) return;
  const int before = r.len - r.n, last = min(r.r0 + kRows, r.rows) - 1;
  const int limit = uniform(max(0, before + last / a.G + 1));
  const Range kr = range_at(limit, KT, r.per, split);
  if (split >= kr.ranges) return;

  // this wave's rows
  const int w0 = r.r0 + 32 * wave, row = min(w0 + col, r.rows - 1);
  const int vis = before + row / a.G + 1;
  const int w_all = before + min(w0, r.rows - 1) / a.G + 1;                                     // keys all its rows see
  const int w_any = w0 < r.rows ? before + min(w0 + 31, r.rows - 1) / a.G + 1 : 0;               // keys any of them sees

  h8 qh[KS], ql[KS];
  float fix = 1.f;  // what a row's own power of two leaves to make up for
  bool fixes;       // whether any row of the wave has one
  {
    const float *q = a.q + (size_t)(r.first + row / a.G) * a.ldq + (size_t)(head * a.G + row % a.G) * D + 8 * half;
    float amax = 0.f;
    float x[KS][8];
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(q + 16 * s + j);
        x[s][j] = v.x * a.scale; x[s][j + 1] = v.y * a.scale; x[s][j + 2] = v.z * a.scale; x[s][j + 3] = v.w * a.scale;
#pragma unroll
        for (int i = 0; i < 4; ++i) amax = fmaxf(amax, finite_abs(x[s][j + i]));
      }
    amax = max_half(amax);
    float up = 1 << kQ;
    const bool own = amax != 0.f && (amax >= 128.f || amax < 0x1p-9f);
    if (own) {
      float down;
      row_factor(amax, up, down);
      fix = down * (1 << kQ);
    }
    fixes = __any(own);
#pragma unroll
    for (int s = 0; s < KS; ++s) pieces8(x[s], up, qh[s], ql[s]);
  }

  // this thread's share: 16 bytes of key kk, and 4 of values 4 vq .. 4 vq + 3
  const int kk = threadIdx.x / (D / 32), kp = threadIdx.x % (D / 32);
  const int vq = threadIdx.x / (D / 8), vb = threadIdx.x % (D / 8);
  const int32_t *table = a.table + (size_t)r.b * a.width;
  const int mask = (1 << a.c.shift) - 1;
  const size_t val = (size_t)a.c.heads << a.c.shift;
  auto page_of = [&](int key) {
    int id = -1;
    if (key < limit) id = table[key >> a.c.shift];
    return (unsigned)id < (unsigned)a.c.pages ? id : -1;
  };
  auto load = [&](int u, int idk, int idv, Codes &x) {
    const size_t vk = (((size_t)max(idk, 0) * 2 * a.c.heads + head) << a.c.shift) + ((u * KT + kk) & mask);
    const size_t vv = (((size_t)max(idv, 0) * 2 * a.c.heads + head) << a.c.shift) + val + ((u * KT + 4 * vq) & mask);
    x.k = *reinterpret_cast<const u4 *>(a.c.codes + vk * (D / 2) + 16 * kp);
    x.wk = a.c.words[vk];
    const uint8_t *v = a.c.codes + vv * (D / 2) + 4 * vb;
#pragma unroll
    for (int i = 0; i < 4; ++i) x.v[i] = *reinterpret_cast<const uint32_t *>(v + i * (D / 2));
    x.wv = *reinterpret_cast<const u4 *>(a.c.words + vv);
  };
  const Masks m = masks();
  // Widened into a stage.  A key that is not there scores -infinity with a
  // weight of nothing.
  auto widen = [&](int u, int idk, int idv, const Codes &x, St &st) {
    // (places in LDS formed anew: kept through the loop they would not fit the
    // registers)
    int thread = threadIdx.x;
    asm volatile("" : "+v"(thread));
    const int kk = thread / (D / 32), kp = thread % (D / 32), vq = thread / (D / 8), vb = thread % (D / 8);
    {
      const Zero z = zero_of(x.wk & 15u, x.wk & 15u);
#pragma unroll
      for (int s = 0; s < 4; ++s) st.k[kk * St::CK + 4 * kp + s] = widen8(x.k[s], m, z);
      if (kp == 0) reinterpret_cast<float *>(st.sk)[kk] = idk >= 0 && u * KT + kk < limit ? scale_of(x.wk) * (1.f / (1 << kQ)) : 0.f;
    }
    const Zero z01 = zero_of(x.wv.x & 15u, x.wv.y & 15u), z23 = zero_of(x.wv.z & 15u, x.wv.w & 15u);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const uint32_t sel = 0x0C040C00u + 0x00010001u * b;
      const uint32_t t01 = __builtin_amdgcn_perm(x.v.y, x.v.x, sel), t23 = __builtin_amdgcn_perm(x.v.w, x.v.z, sel);
      const h2 l01 = widen_lo(t01, m, z01), l23 = widen_lo(t23, m, z23), h01 = widen_hi(t01, m, z01), h23 = widen_hi(t23, m, z23);
      // chunk of keys 16s + 4h + i and 16s + 8 + 4h + i, i < 4: quad vq is its half
      // (vq >> 1) & 1
      const int chunk = 2 * (vq >> 2) + (vq & 1), second = vq >> 1 & 1, row = 2 * b * (D / 8) + vb;
      reinterpret_cast<h4 *>(&st.v[row * St::CV + chunk])[second] = h4{l01.x, l01.y, l23.x, l23.y};
      reinterpret_cast<h4 *>(&st.v[(row + D / 8) * St::CV + chunk])[second] = h4{h01.x, h01.y, h23.x, h23.y};
    }
    if (vb < 4) {
      const int t = 4 * vq + vb;
      const uint32_t w = vb == 0 ? x.wv.x : vb == 1 ? x.wv.y : vb == 2 ? x.wv.z : x.wv.w;
      const bool there = idv >= 0 && u * KT + t < limit;
      float e, inv;
      exponent_of(w, e, inv);
      reinterpret_cast<float *>(st.ex)[t] = there ? e : -__builtin_inff();
      reinterpret_cast<float *>(st.fr)[t] = there ? scale_of(w) * inv : 0.f;
      reinterpret_cast<float *>(st.ie)[t] = there ? inv : 0.f;
    }
  };

  f16v o[DT];
#pragma unroll
  for (int j = 0; j < DT; ++j)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[j][e] = 0.f;
  float M = kNone, l = 0.f;

  Codes x;
  int idk = -1, idv = -1, nk = -1, nv = -1;
  if (kr.u0 < kr.u1) {
    idk = page_of(kr.u0 * KT + kk);
    idv = page_of(kr.u0 * KT + 4 * vq);
    load(kr.u0, idk, idv, x);
    nk = page_of((kr.u0 + 1) * KT + kk);
    nv = page_of((kr.u0 + 1) * KT + 4 * vq);
    widen(kr.u0, idk, idv, x, stage[0]);
  }
  __syncthreads();
  for (int u = kr.u0; u < kr.u1; ++u) {
    const St &st = stage[(u - kr.u0) & 1];
    if (u + 1 < kr.u1) {
      idk = nk;
      idv = nv;
      load(u + 1, idk, idv, x);
      nk = page_of((u + 2) * KT + kk);
      nv = page_of((u + 2) * KT + 4 * vq);
    }
    // A product's operands are asked for well before it (the compiler would ask right in front and wait): keys' first two
    // chunks while the keys before are at work, the others before the first product, values before the weights.
    h8 first[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) first[j] = (&st.k[col * St::CK + half])[2 * j];
#pragma unroll 1
    for (int kt = 0; kt < KT / 32; ++kt) {
      const int key0 = u * KT + 32 * kt;
      if (key0 >= w_any) break;
      const h8 *kb = &st.k[(32 * kt + col) * St::CK + half], *vb0 = &st.v[col * St::CV + 4 * kt + half];
      const int q0 = 8 * kt + half;  // quads of keys: register 4b + i is key 4 (q0 + 2b) + i
      h8 kf[KS];
#pragma unroll
      for (int j = 0; j < KS; ++j) kf[j] = j < 2 ? first[j] : kb[2 * j];
      __builtin_amdgcn_sched_barrier(0);
      f16v s;
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e] = 0.f;
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        s = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf[j], qh[j], s, 0, 0, 0);
        s = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf[j], ql[j], s, 0, 0, 0);
      }
      const h8 *next = kb + (kt + 1 < KT / 32 ? 32 * St::CK : 0);  // (behind the last: once more, unused)
#pragma unroll
      for (int j = 0; j < 2; ++j) first[j] = next[2 * j];
      if (fixes) {
        asm volatile("; rows with a factor of their own");
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] *= fix;
      }
      float top = -__builtin_inff();
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const f4 sk = st.sk[q0 + 2 * b], ex = st.ex[q0 + 2 * b];
#pragma unroll
        for (int i = 0; i < 4; ++i) s[4 * b + i] = fmaf(s[4 * b + i], sk[i], ex[i]);
      }
      f4 fr[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) fr[b] = st.fr[q0 + 2 * b];
      if (key0 + 32 > w_all) {
        asm volatile("; keys behind a query");  // (a branch: most tiles have none)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const bool no = key0 + 8 * (e >> 2) + 4 * half + (e & 3) >= vis;
          s[e] = no ? -__builtin_inff() : s[e];
          // (a weight of exactly nothing, times a value that may not be finite)
          fr[e >> 2][e & 3] = no ? 0.f : fr[e >> 2][e & 3];
        }
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, s[e]);
      top = max_half(top);
      if (__any(top > M + (kLift + kSlack))) {
        // (only the rows that need it: a row's rounding does not go by its neighbours)
        const float up = top > M + (kLift + kSlack) ? top - kLift : M, f = exp2_fast(M - up);
        M = up;
        l *= f;
#pragma unroll
        for (int j = 0; j < DT; ++j) o[j] *= f;
      }
      h8 vf[2][DT];
#pragma unroll
      for (int j = 0; j < DT; ++j) vf[0][j] = vb0[32 * j * St::CV];
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        u4 ph, pl;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const f4 ie = st.ie[q0 + 4 * ks + 2 * b];
          float w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p = exp2_fast(s[8 * ks + 4 * b + i] - M);
            w[i] = p * fr[2 * ks + b][i];
            l = fmaf(p, ie[i], l);
          }
          uint32_t h0, h1, l0, l1;
          pieces2(w[0], w[1], h0, l0);
          pieces2(w[2], w[3], h1, l1);
          ph[2 * b] = h0; ph[2 * b + 1] = h1;
          pl[2 * b] = l0; pl[2 * b + 1] = l1;
        }
        if (ks == 0) {
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int j = 0; j < DT; ++j) vf[1][j] = vb0[32 * j * St::CV + 2];
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int j = 0; j < DT; ++j) {
          o[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[ks][j], __builtin_bit_cast(h8, ph), o[j], 0, 0, 0);
          o[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[ks][j], __builtin_bit_cast(h8, pl), o[j], 0, 0, 0);
        }
      }
    }
    if (u + 1 < kr.u1) widen(u + 1, idk, idv, x, stage[(u + 1 - kr.u0) & 1]);
    __syncthreads();
  }

  l += __shfl_xor(l, 32);
  // (formed anew: kept through the loop they would not fit the registers)
  int thread = threadIdx.x;
  asm volatile("" : "+v"(thread));
  store_rows<D>(a, r, item, head, kr.ranges, wave, thread & 31, thread >> 5 & 1, o, M, l);
}

// The ranges' sums of a tile's rows joined: D / 4 threads a row.  Workgroups take every so many tiles (beside single
// tokens there are far fewer than planned for).
template <int D>
__global__ __launch_bounds__(256) void attn_join_tiles_kernel(AttnArgs a) {
  constexpr int COLS = D / 4;
  const int stride = gridDim.x / a.c.heads, head = blockIdx.x % a.c.heads;
  const int rr = blockIdx.y * (256 / COLS) + threadIdx.x / COLS, c = threadIdx.x % COLS;
  for (int tile = blockIdx.x / a.c.heads; tile < a.tiles; tile += stride) {
    Rows r;
    int unused;
    if (!find_rows<kRows, false>(a, tile, Stage<D>::KT, r, unused)) return;
    const int last = min(r.r0 + kRows, r.rows) - 1, rw = r.r0 + rr;
    const int limit = uniform(max(0, r.len - r.n + last / a.G + 1));
    const int ranges = range_at(limit, Stage<D>::KT, r.per, 0).ranges;
    // (more items than there are only where cu_q does not increase)
    if (ranges > 1 && rw <= last && r.item0 + (ranges - 1) * r.stride < a.items) {
      const size_t step = (size_t)r.stride * a.c.heads * kRows * (D + 4);
      const float *part = a.part + (((size_t)r.item0 * a.c.heads + head) * kRows + rr) * (D + 4);
      float top = kNone;
      for (int t = 0; t < ranges; ++t) top = fmaxf(top, part[t * step + D]);
      f4 v = {0.f, 0.f, 0.f, 0.f};
      float sum = 0.f;
#pragma unroll 4
      for (int t = 0; t < ranges; ++t) {
        const float f = exp2_fast(part[t * step + D] - top);
        sum += f * part[t * step + D + 1];
        v += *reinterpret_cast<const f4 *>(part + t * step + 4 * c) * f;
      }
      *reinterpret_cast<f4 *>(a.out + ((size_t)(r.first + rw / a.G) * a.Hq + head * a.G + rw % a.G) * D + 4 * c) = v * inv_sum(sum);
    }
  }
}

}  // namespace

template <int D>
hipError_t launch_tiles(const AttnArgs &a, hipStream_t stream) {
  constexpr size_t lds = 2 * sizeof(Stage<D>);
  const hipError_t s =
      hipFuncSetAttribute(reinterpret_cast<const void *>(attn_tiles_kernel<D>), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (s != hipSuccess) return s;
  hipLaunchKernelGGL(attn_tiles_kernel<D>, dim3((unsigned)(a.items * a.c.heads)), dim3(64 * kWaves), lds, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int most = (512 + a.c.heads - 1) / a.c.heads;
  hipLaunchKernelGGL(attn_join_tiles_kernel<D>, dim3((unsigned)((a.tiles < most ? a.tiles : most) * a.c.heads), kRows * D / 1024), dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_attn_tiles(const AttnArgs &a, hipStream_t stream) {
  return a.c.D == 128 ? launch_tiles<128>(a, stream) : launch_tiles<64>(a, stream);
}

}  // namespace aq
