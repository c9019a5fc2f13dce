// Attention over the 4-bit cache for few query rows (single tokens, short
// chunks).  Long contexts are bound by the cache's bytes: 64 sequences of 8000 tokens, 32 query heads over 8
// of 128, 557 MB, take 111 us replayed alone (5.0 TB/s) and 121 in a layer (4.6; a large copy moves 4.4 to 4.8).  Short ones are bound by a workgroup's
// chain (us of its 11 for one unit of keys: place 1, pages and codes 2.2, q 1, digits 1, scores, softmax
// and values 2, the waves' sums 1.6): 64 sequences of 256 tokens 10 us, of 257 15, one of 1500 8 and the join 4.
//
// A workgroup takes up to QC rows (4, 8 or 16) of one sequence and key/value head
// and a range of its keys; its four waves take 64 keys each in turn and meet at
// the end.  A wave forms S^T = K Q^T (16 keys x 16 columns a tile), whose
// registers are, as they stand, the weights' operand of O^T = V^T P^T: the order
// of the keys in that product is free, and the values' codes are loaded in the
// order that the weights have.  So nothing passes through LDS but the waves' sums
// at the end, and the codes widen in registers:
//  * a key's go to bytes, by one AND and one shift per four, for the INT8 products: q is
//    taken as four signed digits of eight bits, whose sums are exact; the zero point leaves as z sum(q)
//    behind the product, in whole numbers too.  A feature is off by at most 2^-30 of its row's largest:
//    with three digits, 2^-22 of it, a feature 30 times the others cost the others so much that the output was off by
//    3e-6 in norm, where FP32 products leave 4e-7 and four digits 1.7e-7, at 2 to 4% more time (48 sequences 26.7 -> 28.0 us,
//    64 of 8000 tokens 110.6 -> 111.5);
//  * a value's go to FP16: 0x6400 | c is 1024 + c, and 0x6400 | 16 c is 1024 + 16 c, so that
//    a pair takes an and-or and a packed addition that takes the zero point off
//    (behind the product, sums over long contexts would cancel).
// (As the FP16 subnormals c 2^-24, which the matrix instructions take, codes would need an AND
// alone; but the sums then keep some 7 bits less, 2e-6 against 1e-7.)
//
// With QC < 16 only QC of a tile's 16 columns are rows.  The scores of 16 / QC tiles
// are gathered into one register's lanes (lanes of a row of 16 exchange by DPP at
// no more than a move), so that the softmax and the words' decoding are done once
// per score and not 16 / QC times, and go back for the product with the values,
// where the columns QC .. 2 QC - 1 take the weights' low pieces: one product in place of
// two, added up once at the end.
//
// Long contexts are cut into ranges, a workgroup each, whose sums a second
// launch joins.

#include "aq_attn.h"
#include "aq_device.h"

namespace aq {
namespace {

constexpr int kUnit = 256;  // keys that a workgroup's waves take in a turn

// A move between the lanes of each row of 16: lane n takes lane (n - N) & 15's
// value in the banks (lanes 4b .. 4b + 3) of BANKS, and keeps `old` elsewhere.
template <int N, int BANKS>
__device__ __forceinline__ uint32_t turn(uint32_t old, uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)x, N & 15 ? 0x120 + (N & 15) : 0xE4, 0xF, BANKS, false);
}
// Lane N of each row of 16 for the whole row.
template <int N>
__device__ __forceinline__ uint32_t from_lane(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, 0x150 + N, 0xF, 0xF, false);
}
template <int N>
__device__ __forceinline__ float max_turn(float x) {
  return fmaxf(x, __uint_as_float(turn<N, 15>(0, __float_as_uint(x))));
}
// floor(x + 1/2): the nearest whole number in one instruction.
__device__ __forceinline__ int nearest(float x) {
  int r;
  asm("v_cvt_rpi_i32_f32 %0, %1" : "=v"(r) : "v"(x));
  return r;
}

// What a wave holds of 64 keys, tiles t of 16; lane column col and group g.
template <int QC>
struct Words { u4 k[QC / 4], v[QC / 4]; };    // of keys 16 (16/QC p + col/QC) + 4g + i
template <int D, int QC>
struct Keys {
  uint32_t k[4][D / 32];  // D/4 features of key 16t + col
  uint32_t v[4][4];       // D/16 features of keys 16t + 4g + i
  Words<QC> w;
};

template <int D, int QC>
__global__ __launch_bounds__(256, QC == 16 ? 2 : 3) void attn_rows_kernel(AttnArgs a) {
  constexpr int KI = D / 64, DT = D / 16, SETS = QC / 4, SP = 16 / QC;
  constexpr int LD = D + 4;
  __shared__ float so[4][QC][LD];
  __shared__ float sm[4][QC], sl[4][QC];
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int qc = col % QC, sub = col / QC;
  const int item = blockIdx.x / a.c.heads, head = blockIdx.x - item * a.c.heads;
  Rows r;
  int split = 0;
  if (a.searched) {
    if (!find_rows<QC, true>(a, item, kUnit, r, split)) return;
  } else {
    split = item / a.tiles;
    single_rows<QC>(a, item - split * a.tiles, kUnit, r);
  }
  const int before = r.len - r.n;  // keys in front of the sequence's first query
  const int row = min(r.r0 + qc, r.rows - 1), last = min(r.r0 + QC, r.rows) - 1;
  const int vis = before + row / a.G + 1;  // keys that this lane's row sees
  const int limit = uniform(max(0, before + last / a.G + 1)), all = uniform(before + r.r0 / a.G + 1);
  const Range kr = range_at(limit, kUnit, r.per, split);
  if (split >= kr.ranges) return;

  // pages of 16 turns at a time, lane 4j + t that of tile t in turn j; -1 where no
  // key is visible or the table has no page
  const int32_t *table = a.table + (size_t)r.b * a.width;
  const int mask = (1 << a.c.shift) - 1;
  int ids = -1, u_ids = kr.u0 - 16;
  auto pages = [&](int u, int (&id)[4]) {
    if (u - u_ids >= 16) {
      u_ids = u;
      const int key = (u + (lane >> 2)) * kUnit + wave * 64 + 16 * (lane & 3);
      ids = -1;
      if (key < limit) ids = table[key >> a.c.shift];
      if ((unsigned)ids >= (unsigned)a.c.pages) ids = -1;
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) id[t] = __builtin_amdgcn_readlane(ids, 4 * (u - u_ids) + t);
  };
  // (a page that is not there reads page 0, in bounds and unused)
  const size_t page_vec = (size_t)2 * a.c.heads << a.c.shift, val = page_vec / 2;  // vectors of a page; of its keys
  const uint32_t k_off = col * (D / 2) + g * (D / 8), v_off = 4 * g * (D / 2) + col * (D / 32);
  auto vector = [&](int u, int t, int id) {
    size_t at = (size_t)(uint32_t)max(id, 0) * page_vec + ((size_t)head << a.c.shift) + ((u * kUnit + wave * 64 + 16 * t) & mask);
    asm("" : "+s"(at));  // (kept in scalar registers)
    return at;
  };
  Keys<D, QC> x;
  int id[4];
  auto load_k = [&](int u) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint8_t *k = a.c.codes + vector(u, t, id[t]) * (D / 2);
      if constexpr (D == 128) {
        const u4 w = *reinterpret_cast<const u4 *>(k + k_off);
        x.k[t][0] = w.x; x.k[t][1] = w.y; x.k[t][2] = w.z; x.k[t][3] = w.w;
      } else {
        const u2 w = *reinterpret_cast<const u2 *>(k + k_off);
        x.k[t][0] = w.x; x.k[t][1] = w.y;
      }
    }
  };
  auto load_v = [&](int u) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint8_t *v = a.c.codes + (vector(u, t, id[t]) + val) * (D / 2);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x.v[t][i] = D == 128 ? *reinterpret_cast<const uint32_t *>((v + v_off) + i * (D / 2))
                             : *reinterpret_cast<const uint16_t *>((v + v_off) + i * (D / 2));
    }
  };
  auto load_w = [&](int u) {
#pragma unroll
    for (int p = 0; p < SETS; ++p) {
      // the vectors of this lane's tile
      size_t at;
      if constexpr (SP == 1) {
        at = vector(u, p, id[p]);
      } else {
        const int mine = __shfl(ids, 4 * (u - u_ids) + SP * p + sub);
        at = (size_t)max(mine, 0) * page_vec + ((size_t)head << a.c.shift) + ((u * kUnit + wave * 64 + 16 * (SP * p + sub)) & mask);
      }
      x.w.k[p] = *reinterpret_cast<const u4 *>(a.c.words + at + 4 * g);
      x.w.v[p] = *reinterpret_cast<const u4 *>(a.c.words + val + at + 4 * g);
    }
  };

  if (kr.u0 < kr.u1) {
    pages(kr.u0, id);
    load_k(kr.u0);
    load_w(kr.u0);
    load_v(kr.u0);
  }

  // q as whole numbers n below 2^30 of four signed digits, in the order of a key's bytes: features
  // 0 2 4 6 1 3 5 7 of each eight.  n + 0x80808080 has the digits, each 128 more, as its bytes.
  v4i qd[4][KI];
  int sum_hi, sum_lo;  // the sums of n's upper two digits and of its lower two, negated
  float rf;
  {
    const float *q = a.q + (size_t)(r.first + row / a.G) * a.ldq + (size_t)(head * a.G + row % a.G) * D + g * (D / 4);
    float y[KI][16];
    uint32_t top = 0;  // (as whole numbers magnitudes keep their order, with infinity and NaN behind)
#pragma unroll
    for (int s = 0; s < KI; ++s)
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(q + 16 * s + j);
        y[s][j] = v.x; y[s][j + 1] = v.y; y[s][j + 2] = v.z; y[s][j + 3] = v.w;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(y[s][j + i]) & 0x7FFFFFFFu);
      }
    top = max_halves(top);
    const bool bad = top >= 0x7F800000u;  // a row that is not finite: NaN scores
    const int up = bad ? -256 : 156 - (int)(top >> 23);  // the largest is 2^29 .. 2^30 times 2^-up
    rf = bad ? __uint_as_float(0x7FC00000u) : __builtin_ldexpf(a.scale, -up);
    int digits[4] = {};
#pragma unroll
    for (int s = 0; s < KI; ++s)
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        uint32_t n[4];  // bytes j .. j + 3: features f, f + 2, f + 4, f + 6
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int f = 8 * (j >> 3) + (j & 4 ? 1 : 0) + 2 * i;
          n[i] = (uint32_t)nearest(__builtin_ldexpf(y[s][f], up)) + 0x80808080u;
        }
        const uint32_t a = __builtin_amdgcn_perm(n[1], n[0], 0x05010400u), b = __builtin_amdgcn_perm(n[3], n[2], 0x05010400u);
        const uint32_t c = __builtin_amdgcn_perm(n[1], n[0], 0x07030602u), d = __builtin_amdgcn_perm(n[3], n[2], 0x07030602u);
        qd[0][s][j >> 2] = (int)(__builtin_amdgcn_perm(d, c, 0x07060302u) ^ 0x80808080u);
        qd[1][s][j >> 2] = (int)(__builtin_amdgcn_perm(d, c, 0x05040100u) ^ 0x80808080u);
        qd[2][s][j >> 2] = (int)(__builtin_amdgcn_perm(b, a, 0x07060302u) ^ 0x80808080u);
        qd[3][s][j >> 2] = (int)(__builtin_amdgcn_perm(b, a, 0x05040100u) ^ 0x80808080u);
#pragma unroll
        for (int i = 0; i < 4; ++i) digits[i] = __builtin_amdgcn_sdot4(qd[i][s][j >> 2], 0x01010101, digits[i], false);
      }
    sum_hi = -sum_halves(digits[0] * 256 + digits[1]);
    sum_lo = -sum_halves(digits[2] * 256 + digits[3]);
  }
  const Masks m = masks();

  f4 o[DT];
#pragma unroll
  for (int j = 0; j < DT; ++j) o[j] = f4{0.f, 0.f, 0.f, 0.f};
  float M = kNone, l = 0.f;

  // A unit: the next one's keys are asked for once the scores no longer need this one's, its words and values
  // at the end (a second set of registers instead holds no more than two workgroups to a CU: 30.0 us
  // against 27.2 for 48 sequences, 50 against 43 for 256 of 256 keys).  Behind the last unit it is asked for once
  // more: a branch around the loads would have the compiler wait for all of them.
  auto turn_of = [&](int u) {
    const int key0 = u * kUnit + wave * 64, next = min(u + 1, kr.u1 - 1);
    const Words<QC> &w = x.w;
    // scores of 16 keys x 16 columns a tile: the upper two digits' sums and the lower two's, below 2^26; a set's
    // tiles gathered, register (p, i) of lane (sub, qc, g) key 16 (SP p + sub) + 4g + i
    float d[SETS][4], inv[SETS][4];
#pragma unroll
    for (int p = 0; p < SETS; ++p) {
      v4i s1[SP], s0[SP];
#pragma unroll
      for (int t = 0; t < SP; ++t) {
        v4i c[KI], up = {0, 0, 0, 0};
        s1[t] = s0[t] = up;
#pragma unroll
        for (int j = 0; j < KI; ++j) {
          const uint32_t a0 = x.k[SP * p + t][2 * j], a1 = x.k[SP * p + t][2 * j + 1], by = 0x0F0F0F0Fu;
          c[j] = v4i{(int)(a0 & by), (int)(a0 >> 4 & by), (int)(a1 & by), (int)(a1 >> 4 & by)};
          up = __builtin_amdgcn_mfma_i32_16x16x64_i8(c[j], qd[0][j], up, 0, 0, 0);
          s1[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(c[j], qd[1][j], s1[t], 0, 0, 0);
        }
        s1[t] += up << 8;
        up = v4i{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < KI; ++j) {
          up = __builtin_amdgcn_mfma_i32_16x16x64_i8(c[j], qd[2][j], up, 0, 0, 0);
          s0[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(c[j], qd[3][j], s0[t], 0, 0, 0);
        }
        s0[t] += up << 8;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t x1 = (uint32_t)s1[0][i], x0 = (uint32_t)s0[0][i];
        if constexpr (QC == 8) {
          x1 = turn<8, 0xC>(x1, (uint32_t)s1[1][i]);
          x0 = turn<8, 0xC>(x0, (uint32_t)s0[1][i]);
        }
        if constexpr (QC == 4) {
          x1 = turn<12, 8>(turn<8, 4>(turn<4, 2>(x1, (uint32_t)s1[1][i]), (uint32_t)s1[2][i]), (uint32_t)s1[3][i]);
          x0 = turn<12, 8>(turn<8, 4>(turn<4, 2>(x0, (uint32_t)s0[1][i]), (uint32_t)s0[2][i]), (uint32_t)s0[3][i]);
        }
        // less z sum(n), in whole numbers: rows whose features lie on one side of zero lose nothing
        const uint32_t wk = w.k[p][i];
        const int z = (int)(wk & 15u), hi = (int)x1 + __mul24(z, sum_hi), lo = (int)x0 + __mul24(z, sum_lo);
        float e;
        exponent_of(w.v[p][i], e, inv[p][i]);
        d[p][i] = fmaf(fmaf((float)hi, 65536.f, (float)lo) * scale_of(wk), rf, e);
      }
    }
    const bool full = (id[0] | id[1] | id[2] | id[3]) >= 0 && key0 + 64 <= all;
    uint32_t out = 0;  // bit 4p + i: a key that this lane's row does not see
    if (!full) {
#pragma unroll
      for (int p = 0; p < SETS; ++p) {
        int there = id[SP * p];
#pragma unroll
        for (int t = 1; t < SP; ++t) there = sub == t ? id[SP * p + t] : there;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (there < 0 || key0 + 16 * (SP * p + sub) + 4 * g + i >= vis) out |= 1u << (4 * p + i);
          if (out >> (4 * p + i) & 1) d[p][i] = -__builtin_inff();
        }
      }
    }
    pages(next, id);
    load_k(next);
    float top = fmaxf(fmaxf(d[0][0], d[0][1]), fmaxf(d[0][2], d[0][3]));
#pragma unroll
    for (int p = 1; p < SETS; ++p) top = fmaxf(fmaxf(fmaxf(top, d[p][0]), fmaxf(d[p][1], d[p][2])), d[p][3]);
    if constexpr (QC <= 8) top = max_turn<8>(top);
    if constexpr (QC <= 4) top = max_turn<4>(top);
    top = max_halves(top);
    if (__any(top > M + (kLift + kSlack))) {
      // (only the rows that need it: a row's rounding does not go by its neighbours)
      const float up = top > M + (kLift + kSlack) ? top - kLift : M, f = exp2_fast(M - up);
      M = up;
      l *= f;
#pragma unroll
      for (int j = 0; j < DT; ++j) o[j] *= f;
    }
    // weights in two pieces
    uint32_t hi[SETS][2], lo[SETS][2], zz[SETS][2];
#pragma unroll
    for (int p = 0; p < SETS; ++p) {
      float wt[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p2 = exp2_fast(d[p][i] - M);
        float den = p2 * inv[p][i];
        wt[i] = p2 * (scale_of(w.v[p][i]) * inv[p][i]);
        if (!full) {
          const bool no = out >> (4 * p + i) & 1;
          den = no ? 0.f : den;
          wt[i] = no ? 0.f : wt[i];
        }
        l += den;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        pieces2(wt[2 * e], wt[2 * e + 1], hi[p][e], lo[p][e]);
        // the zero points of two keys side by side
        zz[p][e] = __builtin_amdgcn_perm(w.v[p][2 * e + 1], w.v[p][2 * e], 0x0C040C00u) & 0x000F000Fu;
      }
    }
    // values, 32 keys a product
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t bh[4], bl[4], z[4];  // two keys each: tile 2h, then 2h + 1
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = 2 * h + tt, p = t / SP, at = 2 * tt + e;
          const uint32_t H = hi[p][e], L = lo[p][e];
          if constexpr (QC == 16) {
            bh[at] = H;
            bl[at] = L;
            z[at] = zz[p][e];
          } else if constexpr (QC == 8) {
            bh[at] = tt ? turn<0, 0xC>(turn<8, 3>(H, H), L) : turn<8, 0xC>(H, L);
            z[at] = tt ? from_lane<8>(zz[p][e]) : from_lane<0>(zz[p][e]);
          } else {
            bh[at] = t == 0 ? turn<4, 2>(H, L) : t == 1 ? turn<0, 2>(turn<12, 1>(H, H), L)
                   : t == 2 ? turn<12, 2>(turn<8, 1>(H, H), L) : turn<8, 2>(turn<4, 1>(H, H), L);
            z[at] = t == 0 ? from_lane<0>(zz[p][e]) : t == 1 ? from_lane<4>(zz[p][e])
                  : t == 2 ? from_lane<8>(zz[p][e]) : from_lane<12>(zz[p][e]);
          }
        }
      const h8 ph = __builtin_bit_cast(h8, u4{bh[0], bh[1], bh[2], bh[3]});
      h8 pl;
      if constexpr (QC == 16) pl = __builtin_bit_cast(h8, u4{bl[0], bl[1], bl[2], bl[3]});
      // byte b of the tokens' words holds features 2b and 2b + 1
#pragma unroll
      for (int b = 0; b < DT / 2; ++b) {
        h2 c[4], e[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t two =
              __builtin_amdgcn_perm(x.v[2 * h + (q >> 1)][2 * (q & 1) + 1], x.v[2 * h + (q >> 1)][2 * (q & 1)], 0x0C040C00u + 0x00010001u * b);
          c[q] = as_h2((two & m.lo) | 0x64006400u) + as_h2(z[q] | 0xE400E400u);
          e[q] = as_h2((two & m.hi) | 0x64006400u) + as_h2(z[q] << 4 | 0xE400E400u);
        }
        const h8 f0 = join8(c[0], c[1], c[2], c[3]), f1 = join8(e[0], e[1], e[2], e[3]);
        o[2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f0, ph, o[2 * b], 0, 0, 0);
        o[2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f1, ph, o[2 * b + 1], 0, 0, 0);
        if constexpr (QC == 16) {
          o[2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f0, pl, o[2 * b], 0, 0, 0);
          o[2 * b + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f1, pl, o[2 * b + 1], 0, 0, 0);
        }
      }
    }
    load_w(next);
    load_v(next);
  };
#pragma unroll 1
  for (int u = kr.u0; u < kr.u1; ++u) turn_of(u);

  // the four waves' sums
  if constexpr (QC <= 8) l += __uint_as_float(turn<8, 15>(0, __float_as_uint(l)));
  if constexpr (QC <= 4) l += __uint_as_float(turn<4, 15>(0, __float_as_uint(l)));
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (lane < QC) {
    sm[wave][lane] = M;
    sl[wave][lane] = l;
  }
  __syncthreads();
  const float top = fmaxf(fmaxf(sm[0][qc], sm[1][qc]), fmaxf(sm[2][qc], sm[3][qc]));
  const float f = exp2_fast(M - top);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < DT; ++j) {
      // (the low pieces' columns; odd features came 16-fold)
      float x = o[j][i] * (j & 1 ? f * 0.0625f : f);
      if constexpr (QC <= 8) x += __uint_as_float(turn<16 - QC, 15>(0, __float_as_uint(x)));
      if (col < QC) so[wave][col][DT * (4 * g + i) + j] = x;
    }
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
      v *= inv_sum(sum);
      *reinterpret_cast<f4 *>(a.out + ((size_t)(r.first + rw / a.G) * a.Hq + head * a.G + rw % a.G) * D + d) = v;
    } else {
      const size_t at = ((size_t)item * a.c.heads + head) * QC + rr;
      float *part = a.part + at * (D + 4);
      *reinterpret_cast<f4 *>(part + d) = v;
      if (d == 0) {
        part[D] = m;
        part[D + 1] = sum;
      }
    }
  }
}

// The ranges' sums of a row joined, a workgroup per row: every wave finds the
// ranges' factors (lane t that of range t), and the workgroup's 256 / (D/4) groups of
// threads add every so many ranges.
template <int D, int QC>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  constexpr int COLS = D / 4, GROUPS = 256 / COLS;
  __shared__ float sf[64];
  __shared__ f4 sv[GROUPS][COLS];
  const int lane = threadIdx.x & 63, rr = blockIdx.y;
  const int tile = blockIdx.x / a.c.heads, head = blockIdx.x - tile * a.c.heads;
  Rows r;
  int unused;
  if (!a.searched)
    single_rows<QC>(a, tile, kUnit, r);
  else if (!find_rows<QC, false>(a, tile, kUnit, r, unused))
    return;
  const int last = min(r.r0 + QC, r.rows) - 1;
  const int limit = uniform(max(0, r.len - r.n + last / a.G + 1));
  const int ranges = range_at(limit, kUnit, r.per, 0).ranges;
  if (ranges == 1 || rr > last - r.r0 || r.item0 + (ranges - 1) * r.stride >= a.items) return;  // (more only where cu_q does not increase)
  const size_t step = (size_t)r.stride * a.c.heads * QC * (D + 4);
  const float *part = a.part + (((size_t)r.item0 * a.c.heads + head) * QC + rr) * (D + 4);
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
  if (threadIdx.x < 64) sf[lane] = f;
  __syncthreads();
  const int c = threadIdx.x % COLS, g = threadIdx.x / COLS;
  f4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int t = g; t < ranges; t += GROUPS) v += *reinterpret_cast<const f4 *>(part + t * step + 4 * c) * sf[t];
  sv[g][c] = v;
  __syncthreads();
  if (g == 0) {
#pragma unroll
    for (int t = 1; t < GROUPS; ++t) v += sv[t][c];
    const int rw = r.r0 + rr;
    *reinterpret_cast<f4 *>(a.out + ((size_t)(r.first + rw / a.G) * a.Hq + head * a.G + rw % a.G) * D + 4 * c) = v * inv_sum(sum);
  }
}

template <int D, int QC>
hipError_t rows(const AttnArgs &a, hipStream_t stream) {
  hipLaunchKernelGGL((attn_rows_kernel<D, QC>), dim3((unsigned)(a.items * a.c.heads)), dim3(256), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL((attn_join_kernel<D, QC>), dim3((unsigned)(a.tiles * a.c.heads), QC), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_rows(const AttnArgs &a, int qc, hipStream_t stream) {
  if (a.c.D == 128) return qc == 4 ? rows<128, 4>(a, stream) : qc == 8 ? rows<128, 8>(a, stream) : rows<128, 16>(a, stream);
  return qc == 4 ? rows<64, 4>(a, stream) : qc == 8 ? rows<64, 8>(a, stream) : rows<64, 16>(a, stream);
}

}  // namespace aq
