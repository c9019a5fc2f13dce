// A mixture-of-experts layer over packed W4/W8 experts, for few tokens an expert.
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
// read once for up to 32 of its tokens.
//   Up to 16 pairs with h rows of up to 2048 take three launches for a whole layer:
//   (1) logits and INT8 rows; (2) gate/up, whose workgroups choose the experts
//   themselves and find their own expert's pairs; (3) down, whose workgroups
//   quantize the h rows, pass over all pairs' experts for 16 output features and
//   add them up.  The choice is a launch of its own beyond 8 tokens or 256 experts,
//   where the logits are partial sums, and where gate/up has more workgroups than
//   run at once.
//   More pairs or longer rows: down is split over the experts too, and a last
//   launch adds a token's outputs; beyond 8 pairs an expert, and for longer rows, h
//   is quantized by a launch; beyond 512 pairs they are first listed per expert.

#include "aq_quant.h"
#include "aq_route.h"
#include "aq_routed.h"
#include "aq_tile_stream.h"

namespace aq {
namespace {

struct MoeArgs {
  Packed gu, dn;
  RouteArgs rt;  // the layer's router (the fused choice)
  const int8_t *qx;
  const float *sx;
  int32_t *ids;
  float *weights;
  int32_t *lists;  // [0] = number of active experts, then active [E], start [E + 1], pair [P]
  float *h;
  int8_t *qh;
  float *sh;
  float *d;
  float *Y;
  int M, top_k, E, H, I, P;
};

// ---- lists: pairs grouped by expert, written by one workgroup of 1024
// threads (ids: LDS or global).  An id outside 0 .. E-1 belongs to no expert.
// The place of a pair inside its expert's run depends on the order of the
// LDS atomics, its result does not: every pair is one row of an MFMA operand
// and its outputs are its own.
static_assert(AQ_MOE_MAX_EXPERTS == 1024, "one thread per expert");
__device__ __forceinline__ void write_lists(const int32_t *ids, int P, int E, int32_t *__restrict__ lists) {
  __shared__ int cnt[1024], pos[1024];
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
#pragma unroll
  for (int w = 0; w < 15; ++w) {  // (all loads at once)
    s += w < wave ? wsum[w] : 0;
    a += w < wave ? wact[w] : 0;
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

__global__ __launch_bounds__(1024) void moe_lists_kernel(const MoeArgs a) {
  write_lists(a.ids, a.P, a.E, a.lists);
}

// ---- which pairs are mine.  Up to kScanMaxP pairs every workgroup reads the
// ids and finds its expert's pairs by itself (one load round trip, then
// ballots; the lists take a launch and three dependent loads).  Slot s stands
// for the expert of pair s where no earlier pair has it (P <= E), else for
// expert s.  Returns false where there is nothing to do; uniform over the
// workgroup.
// (1600 pairs: 4.9 us for the lists, then gate/up 60 us and down 35; without
// them 67 and 43.)
constexpr int kScanMaxP = 512;
enum { kLists = 0, kScan = 1, kChoose = 2 };

__device__ __forceinline__ bool find_pairs(const MoeArgs &a, const int32_t *ids, int slot, int32_t *own, int lane,
                                           int &e, int &cnt) {
  const bool by_pair = a.P <= a.E;
  e = by_pair ? __builtin_amdgcn_readfirstlane(ids[slot]) : slot;
  if ((unsigned)e >= (unsigned)a.E) return false;
  cnt = 0;
  for (int b = 0; b < a.P; b += 64) {
    const bool hit = b + lane < a.P && ids[b + lane] == e;
    const uint64_t hits = __ballot(hit);
    if (by_pair && cnt == 0 && hits && b + __builtin_ctzll(hits) < slot) return false;
    // every wave writes the same list and reads what it has written itself, so
    // that no barrier is needed
    if (hit) own[cnt + __popcll(hits & ((1ull << lane) - 1ull))] = b + lane;
    cnt += __popcll(hits);
  }
  return cnt > 0;
}

// ---- gate and up: a wave takes 16 features of one active expert (16 gate
// rows and 16 up rows) over one of S ranges of the tile columns; a workgroup
// holds 4 / 4 / 2 / 1 such feature groups for S = 1 / 2 / 4 / 8.  The ranges'
// FP64 sums meet in LDS in increasing order.
constexpr int kChooseMaxM = 8;  // tokens whose experts every gate/up workgroup chooses itself, one wave per token
constexpr int gu_waves(int S) { return S == 1 ? 4 : 8; }

// Whole rows per wave (S == 1): the tokens' codes go through LDS, 512 columns at
// a time, two such chunks deep, so that the four waves fetch them once (200
// tokens, 128 experts of 2048 x 768: 53 us, against 60 with every wave loading
// its own; 32 tokens, 32 experts of 4096 x 1536: 42 against 44; four tile columns
// of weights in flight instead of two: 56 and 44).
constexpr int kXCols = 512, kXStride = kXCols + 16;  // (rows 16 bytes apart in the banks)

template <int BK, int NG, int S>
__device__ __forceinline__ void gate_up_pass(const MoeArgs &a, double (*red)[2][4][64], int8_t *xs, int e, const int32_t *pair,
                                             int b, int cnt, int f, int sp, int lane, int wave) {
  constexpr int ST = 2;                   // pipeline stages: tile columns in flight
  constexpr int EL = S >= 4 ? 1 : 4 / S;  // elements a wave finishes
  const int g = lane >> 4, i16 = lane & 15;
  const int RI = a.I >> 6;
  const int rgate = e * 2 * RI + (f >> 2);
  const int C = a.gu.C, c0 = C * sp / S, c1 = C * (sp + 1) / S;
  const RowMeta mg(a.gu, rgate), mu(a.gu, rgate + RI);
  RowStream<BK> rg(a.gu, mg, f & 3, c0, c1, lane), ru(a.gu, mu, f & 3, c0, c1, lane);
  constexpr bool XLDS = S == 1;
  const int8_t *x[NG];
#pragma unroll
  for (int n = 0; n < NG; ++n)  // tokens past the last repeat it; not stored
    x[n] = a.qx + (size_t)((unsigned)pair[min(b + 16 * n + i16, cnt - 1)] / (unsigned)a.top_k) * a.H;
  int xc = c0;
  struct Stage {
    Tile tg, tu;
    TileX<BK> x[XLDS ? 1 : NG];
  } st[ST];
  auto fetch = [&](Stage &s) __attribute__((always_inline)) {
    rg.fetch(s.tg);
    ru.fetch(s.tu);
    if constexpr (!XLDS) {
#pragma unroll
      for (int n = 0; n < NG; ++n) s.x[n].load(x[n] + min(xc, C - 1) * BK, g);
      ++xc;
    }
  };
  // XLDS: thread: 16 bytes of 2 NG rows, 8 rows apart
  uint32_t xtok[2 * NG];
  v4i xv[2 * NG];
  const int piece = 16 * (threadIdx.x & 31);
  auto load_chunk = [&](int col) __attribute__((always_inline)) {
    int H = a.H;
    asm volatile("" : "+s"(H));  // (the rows' addresses are formed anew: registers)
    const int at = min(col * BK + piece, H - 16);  // columns past the last are not multiplied
#pragma unroll
    for (int i = 0; i < 2 * NG; ++i) xv[i] = load16(a.qx + (uint64_t)xtok[i] * (uint32_t)H + at);
  };
  auto write_chunk = [&](int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2 * NG; ++i)
      *reinterpret_cast<v4i *>(xs + (buf * 16 * NG + 8 * i + (threadIdx.x >> 5)) * kXStride + piece) = xv[i];
    // (LDS writes done; the weights' loads stay open)
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  if constexpr (XLDS) {
#pragma unroll
    for (int i = 0; i < 2 * NG; ++i)
      xtok[i] = (unsigned)pair[min(b + 8 * i + (int)(threadIdx.x >> 5), cnt - 1)] / (unsigned)a.top_k;
    load_chunk(0);
  }
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) fetch(st[i]);
  // element k = sp * EL + i of a lane: token 4g + k, feature i16
  float sxv[NG][EL];
#pragma unroll
  for (int n = 0; n < NG; ++n)
#pragma unroll
    for (int i = 0; i < EL; ++i)
      sxv[n][i] = a.sx[(unsigned)pair[min(b + 16 * n + 4 * g + ((sp * EL + i) & 3), cnt - 1)] / (unsigned)a.top_k];
  double G[NG][4], U[NG][4];
#pragma unroll
  for (int n = 0; n < NG; ++n)
#pragma unroll
    for (int k = 0; k < 4; ++k) G[n][k] = U[n][k] = 0.;
  // SwiGLU of element k of token group n from its two sums
  auto finish = [&](int n, int k, int i, double sg, double su) __attribute__((always_inline)) {
    const int tok = b + 16 * n + 4 * g + k;
    if (tok < cnt) {
      const double s = (double)sxv[n][i];
      sg *= s;
      su *= s;
      a.h[(size_t)pair[tok] * a.I + (f << 4) + i16] = (float)(sg / (1. + exp(-sg)) * su);
    }
    __builtin_amdgcn_sched_barrier(0);  // one exponential at a time: interleaved they spill
  };
  // xop(n): the codes of token group n for the stage's column
  auto multiply = [&](const Stage &s, auto xop) __attribute__((always_inline)) {
    {
      const double sc = (double)scale_of(s.tg);
      const TileOp<BK> w(s.tg);
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const v4i v = tile_product<BK>(w, xop(n), s.tg.is4);
#pragma unroll
        for (int k = 0; k < 4; ++k) G[n][k] = fma((double)v[k], sc, G[n][k]);
      }
    }
    if (NG > 1) __builtin_amdgcn_sched_barrier(0);  // one tile's operands at a time (registers)
    {
      const double sc = (double)scale_of(s.tu);
      const TileOp<BK> w(s.tu);
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const v4i v = tile_product<BK>(w, xop(n), s.tu.is4);
#pragma unroll
        for (int k = 0; k < 4; ++k) U[n][k] = fma((double)v[k], sc, U[n][k]);
      }
    }
  };
  if constexpr (XLDS) {
    constexpr int CPC = kXCols / BK;  // tile columns a chunk
    if (b) __syncthreads();           // the last pass's codes have been read
    write_chunk(0);
    int buf = 0;
#pragma unroll 1
    for (int j = 0; j < C; j += CPC) {
      load_chunk(j + CPC);
      const int8_t *xb = xs + (buf * 16 * NG + i16) * kXStride;
#pragma unroll
      for (int i = 0; i < CPC; ++i) {
        fetch(st[(i + ST - 1) % ST]);
        if (j + i < C)
          multiply(st[i % ST], [&](int n) __attribute__((always_inline)) {
            TileX<BK> t;
            t.load(xb + 16 * n * kXStride + i * BK, g);
            return t;
          });
      }
      buf ^= 1;
      write_chunk(buf);
    }
  } else {
#pragma unroll 1
    for (int j = c0; j < c1; j += ST) {
#pragma unroll
      for (int i = 0; i < ST; ++i) {
        fetch(st[(i + ST - 1) % ST]);
        if (j + i < c1) multiply(st[i], [&](int n) __attribute__((always_inline)) { return st[i].x[n]; });
      }
    }
  }
  if constexpr (S == 1) {
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) finish(n, k, k, G[n][k], U[n][k]);
  } else {
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      if (b + n) __syncthreads();  // the last group's sums have been read
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        red[wave][0][k][lane] = G[n][k];
        red[wave][1][k][lane] = U[n][k];
      }
      __syncthreads();
      if (sp * EL >= 4) continue;
#pragma unroll
      for (int i = 0; i < EL; ++i) {
        const int k = sp * EL + i, w0 = wave - sp;
        double sg = 0., su = 0.;
#pragma unroll
        for (int w = 0; w < S; ++w) {
          sg += red[w0 + w][0][k][lane];
          su += red[w0 + w][1][k][lane];
        }
        finish(n, k, i, sg, su);
      }
    }
  }
}

// Whole rows per wave take up to 32 tokens a pass, in 168 registers (3 waves
// per SIMD); the others 16 in 128.
constexpr bool gu_two(int S) { return S == 1; }

template <int BK, int MODE, int NE, int S>
__global__ __launch_bounds__(gu_waves(S) * 64, gu_two(S) ? 3 : 4) void moe_gate_up_kernel(const MoeArgs a) {
  constexpr int WAVES = gu_waves(S);
  constexpr bool TWO = gu_two(S);
  __shared__ double red[S > 1 ? WAVES : 1][2][4][S > 1 ? 64 : 1];
  __shared__ __align__(16) int8_t xs[S > 1 ? 16 : 2 * 16 * (TWO ? 2 : 1) * kXStride];
  constexpr int kMost = MODE == kLists ? 1 : MODE == kScan ? kScanMaxP : kChooseMaxM * AQ_MOE_MAX_TOP_K;
  __shared__ int32_t ids[kMost], own[kMost];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int e, cnt;
  const int32_t *pair;
  if constexpr (MODE == kLists) {
    if ((int)blockIdx.y >= uload(a.lists)) return;
    e = uload(a.lists + 1 + blockIdx.y);
    const int32_t *start = a.lists + 1 + a.E;
    const int p0 = uload(start + e);
    cnt = uload(start + e + 1) - p0;
    pair = start + a.E + 1 + p0;
  } else {
    if constexpr (MODE == kChoose) {
      // every workgroup makes the same choice; the first one writes it out
      for (int m = wave; m < a.M; m += WAVES) {
        int id;
        float w;
        const bool first = blockIdx.x == 0 && blockIdx.y == 0;
        choose<NE>(a.rt, a.rt.logits + (size_t)m * a.E, lane, first, id, w);
        if (lane < a.top_k) {
          ids[m * a.top_k + lane] = id;
          if (first) {
            a.ids[m * a.top_k + lane] = id;
            a.weights[m * a.top_k + lane] = w;
          }
        }
      }
    } else {
      for (int p = threadIdx.x; p < a.P; p += WAVES * 64) ids[p] = a.ids[p];
    }
    __syncthreads();
    if (!find_pairs(a, ids, blockIdx.y, own, lane, e, cnt)) return;
    pair = own;
  }
  const int f = blockIdx.x * (WAVES / S) + wave / S, sp = wave % S;
  const auto sums = reinterpret_cast<double (*)[2][4][64]>(red);
  constexpr int PASS = TWO ? 32 : 16;
  for (int b = PASS * blockIdx.z; b < cnt; b += PASS * gridDim.z) {
    if (TWO && cnt - b > 16) gate_up_pass<BK, TWO ? 2 : 1, S>(a, sums, xs, e, pair, b, cnt, f, sp, lane, wave);
    else gate_up_pass<BK, 1, S>(a, sums, xs, e, pair, b, cnt, f, sp, lane, wave);
  }
}

// ---- down and combine, up to kRowsMaxP pairs: one workgroup of 16 waves per
// 16 output features, which passes over all the pairs' experts.  An item is
// up to 16 pairs of one expert; items are cut into S column ranges and dealt
// to the waves.  Each (pair, range) leaves its FP32 sums in LDS, and a
// token's are added in the order of its slots and ranges, so neither the
// grouping nor the dealing enters the result.  The workgroup quantizes the
// pairs' h rows itself, one wave per row, under its first weight loads (codes
// in LDS, rows 16 bytes apart in the banks).
// (The layer with this form / with the one for more pairs, microseconds: 8 pairs at 8
// experts of 2048 x 768 21.4 / 23.5, 2 of 2048 x 1024 17.0 / 18.4, 4 of 4096 x 1536
// 24.8 / 27.9; 16 pairs at 15 of 2048 x 768 27.8 / 28.3, at 13 of 4096 x 1536 49.7 /
// 50.4, at 7 of 2048 x 1024 22.4 / 21.8; 20 pairs at 14 of 2560 x 1280, with room made
// for 32, 40.7 / 38.8.)
constexpr int kRowsMaxP = 16;

struct RowsLds {
  float parts[16 * kRowsMaxP * 16];  // [pair][range][16]
  int32_t ids[kRowsMaxP], pair[kRowsMaxP];
  int32_t item_e[kRowsMaxP], item_at[kRowsMaxP], item_n[kRowsMaxP];
  float scale[kRowsMaxP];  // sh * weight of a pair
  int32_t nitems, pad[3];
};
// Column ranges per item, of T items at most (not of those there are: a token's
// order of sums would depend on the other tokens' experts): the cheapest of the
// powers of two for 16 waves, where a (item, range) costs its columns and about 8 columns' time until its
// first weights are there.
__device__ __forceinline__ int rows_split(int T, int C) {
  int best = 1, cost = ((T + 15) / 16) * (C + 8);
#pragma unroll
  for (int s = 2; s <= 16; s <<= 1) {
    const int c = ((T * s + 15) / 16) * ((C + s - 1) / s + 8);
    if (s <= C && c < cost) {
      best = s;
      cost = c;
    }
  }
  return best;
}

// The lane's 4 sums per tile row against NG times 16 token rows (x[n]: the
// lane's row of codes), for one or more consecutive tile rows: their tiles
// follow one another in the packed order, so that a walk simply goes on into
// the next row, its first tiles in flight while the last are multiplied.
// Columns c0 .. c1-1 of one row, or c1 = a multiple of C (c0 = 0) for several.
// XLDS: the codes are in LDS and read as they are needed; otherwise they are
// loaded with the weights.  The constructor issues the first stages.
template <int BK, int NG, bool XLDS>
struct DownPipe {
  static constexpr int ST = NG == 1 || XLDS ? 4 : 2;
  struct Stage {
    Tile t;
    TileX<BK> x[XLDS ? 1 : NG];
  } st[ST];
  RowStream<BK> rs;
  int c0, g, xc;
  __device__ __forceinline__ void fetch(Stage &s, const int8_t *const (&x)[NG]) {
    rs.fetch(s.t);
    if constexpr (!XLDS) {
#pragma unroll
      for (int n = 0; n < NG; ++n) s.x[n].load(x[n] + xc * BK, g);
      xc = xc + 1 == rs.p.C ? 0 : xc + 1;
    }
  }
  __device__ __forceinline__ DownPipe(const Packed &p, const RowMeta &m, int rg, int c0_, int c1, int lane,
                                      const int8_t *const (&x)[NG])
      : rs(p, m, rg, c0_, c1, lane), c0(c0_), g(lane >> 4), xc(c0_) {
#pragma unroll
    for (int i = 0; i < ST - 1; ++i) fetch(st[i], x);
  }
  // emit(row, F) at the end of each tile row
  template <typename E>
  __device__ __forceinline__ void run(const int8_t *const (&x)[NG], E emit) {
    float F[NG][4];
    auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int n = 0; n < NG; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) F[n][k] = 0.f;
    };
    clear();
    const int c1 = rs.c1, C = rs.p.C;
    int col = c0, row = 0;
#pragma unroll 1
    for (int j = c0; j < c1; j += ST) {
#pragma unroll
      for (int i = 0; i < ST; ++i) {
        fetch(st[(i + ST - 1) % ST], x);
        if (j + i < c1) {
          Stage &s = st[i];
          const TileOp<BK> w(s.t);
          const float sc = scale_of(s.t);
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            TileX<BK> xo;
            if constexpr (XLDS) xo.load(x[n] + col * BK, g);
            else xo = s.x[n];
            const v4i v = tile_product<BK>(w, xo, s.t.is4);
#pragma unroll
            for (int k = 0; k < 4; ++k) F[n][k] = fmaf((float)v[k], sc, F[n][k]);
          }
          ++col;
          if (col == C || j + i + 1 == c1) {
            emit(row, F);
            clear();
            ++row;
            col = 0;
          }
        }
      }
    }
  }
};

// One wave quantizes a row of I <= kFuseqMaxI values into LDS (the rule of
// aq_quant_act); the row is read once into registers.
constexpr int kFuseqMaxI = 2048;
struct HRow {
  float4 v[kFuseqMaxI / 256];
  __device__ __forceinline__ void load(const float *h, int I, int lane) {
    const float4 *row = reinterpret_cast<const float4 *>(h);
#pragma unroll
    for (int i = 0; i < kFuseqMaxI / 256; ++i)
      if (256 * i < I) v[i] = row[min(lane + 64 * i, (I >> 2) - 1)];  // uniform: only the loads that the row has
  }
  // codes into LDS; returns the scale
  __device__ __forceinline__ float quantize(int I, int8_t *codes, int lane) const {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < kFuseqMaxI / 256; ++i)
      if (256 * i < I) amax = max(amax, abs_bits4(v[i]));
    const double sc = row_scale(wave_max_rows_u32(amax));
    const float inv = (float)(1.0 / sc);
    uint32_t *out = reinterpret_cast<uint32_t *>(codes);
#pragma unroll
    for (int i = 0; i < kFuseqMaxI / 256; ++i)
      if (lane + 64 * i < (I >> 2)) out[lane + 64 * i] = codes4_fast(v[i], sc, inv);
    return (float)sc;
  }
};

template <int BK>
__global__ __launch_bounds__(1024) void moe_down_rows_kernel(const MoeArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  RowsLds &s = *reinterpret_cast<RowsLds *>(smem);
  int8_t *codes = reinterpret_cast<int8_t *>(smem + sizeof(RowsLds));
  const int cstride = a.I + 16;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  const int P = a.P;
  // ---- items: the first wave counts the pairs before and of each pair's
  // expert
  if (wave == 0) {
    const int e = lane < P ? a.ids[lane] : -1;
    const bool valid = (unsigned)e < (unsigned)a.E;
    int before = 0, rank = 0, all = 0;
#pragma unroll
    for (int j = 0; j < kRowsMaxP; ++j) {
      const int o = __builtin_amdgcn_readlane(valid ? e : -1, j);
      if (j < P && o >= 0) {
        before += o < e;
        all += o == e;
        rank += o == e && j < lane;
      }
    }
    const uint64_t first = __ballot(valid && rank == 0);  // (at most 16 pairs: one item per expert)
    if (lane < P) s.ids[lane] = valid ? e : -1;
    if (valid) s.pair[before + rank] = lane;
    if (valid && rank == 0) {
      const int at = __popcll(first & ((1ull << lane) - 1ull));
      s.item_e[at] = e;
      s.item_at[at] = before;
      s.item_n[at] = all;
    }
    if (lane == 0) s.nitems = __popcll(first);
  }
  __syncthreads();
  const int T = __builtin_amdgcn_readfirstlane(s.nitems), C = a.dn.C;
  const int S = rows_split(min(P, a.E), C);
  const int rg = blockIdx.x & 3;
  // work w: item w / S, column range w % S
  struct Work {
    int e, at, n, sp, c0, c1;
  };
  auto work = [&](int w) __attribute__((always_inline)) {
    const int it = w / S, sp = w - it * S;
    return Work{__builtin_amdgcn_readfirstlane(s.item_e[it]), __builtin_amdgcn_readfirstlane(s.item_at[it]),
                __builtin_amdgcn_readfirstlane(s.item_n[it]), sp, C * sp / S, C * (sp + 1) / S};
  };
  auto meta = [&](const Work &k) __attribute__((always_inline)) {
    return RowMeta(a.dn, k.e * (a.H >> 6) + ((int)blockIdx.x >> 2));
  };
  auto codes_of = [&](const Work &k) __attribute__((always_inline)) {
    return codes + (size_t)s.pair[k.at + min(i16, k.n - 1)] * cstride;
  };
  typedef DownPipe<BK, 1, true> Pipe;
  auto finish = [&](Pipe &pipe, const Work &k, const int8_t *const (&x)[1]) __attribute__((always_inline)) {
    pipe.run(x, [&](int, const float (&F)[1][4]) __attribute__((always_inline)) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (4 * g + q < k.n) {
          const int p = s.pair[k.at + 4 * g + q];
          s.parts[(p * S + k.sp) * 16 + i16] = F[0][q] * s.scale[p];
        }
    });
  };
  // the wave's row of h (its loads go out with the first weights')
  const bool mine = wave < P && s.ids[min(wave, P - 1)] >= 0;
  HRow hr;
  auto quantize = [&]() __attribute__((always_inline)) {
    if (mine) {
      const float sc = hr.quantize(a.I, codes + (size_t)wave * cstride, lane);
      if (lane == 0) s.scale[wave] = sc * a.weights[wave];
    }
    // (LDS writes done; the weights' loads stay open)
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  if (wave < T * S) {
    const Work k = work(wave);
    const RowMeta m = meta(k);
    if (mine) hr.load(a.h + (size_t)wave * a.I, a.I, lane);
    const int8_t *x[1] = {codes_of(k)};
    Pipe pipe(a.dn, m, rg, k.c0, k.c1, lane, x);
    quantize();
    finish(pipe, k, x);
  } else {
    if (mine) hr.load(a.h + (size_t)wave * a.I, a.I, lane);
    quantize();
  }
  for (int w = wave + 16; w < T * S; w += 16) {
    const Work k = work(w);
    const int8_t *x[1] = {codes_of(k)};
    Pipe pipe(a.dn, meta(k), rg, k.c0, k.c1, lane, x);
    finish(pipe, k, x);
  }
  __syncthreads();
  for (int o = tid; o < a.M * 16; o += 1024) {
    const int m = o >> 4, i = o & 15;
    float y = 0.f;
#pragma unroll 4
    for (int k = 0; k < a.top_k; ++k) {
      const int p = m * a.top_k + k;
      float v = s.parts[p * S * 16 + i];
      for (int q = 1; q < S; ++q) v += s.parts[(p * S + q) * 16 + i];
      y += s.ids[p] >= 0 ? v : 0.f;  // (sums of a pair without an expert hold anything)
    }
    a.Y[(size_t)m * a.H + blockIdx.x * 16 + i] = y;
  }
}

// ---- down, more pairs: one workgroup of 4 waves per TR consecutive tile rows
// of one active expert, a wave per 16 rows of each over all tile columns, 32
// pairs a pass.  Their codes come
//   kQuantize: from h, which the workgroup quantizes into LDS,
//   kCopy:     from qh, copied into LDS,
//   kDirect:   from qh as the tiles are multiplied (rows too long for LDS).
// (1600 pairs over 128 experts of 2048 x 768: kCopy 34.7 us and 5 us for the
// quantizer's launch, kQuantize 45.8 us, kDirect 45 and 5.)
enum { kQuantize = 0, kCopy = 1, kDirect = 2 };
template <int BK, int SRC, bool SCAN>
__global__ __launch_bounds__(256, 4) void moe_down_kernel(const MoeArgs a, int TR, int held) {
  extern __shared__ __align__(16) int8_t codes[];
  __shared__ int32_t ids[SCAN ? kScanMaxP : 1], own[SCAN ? kScanMaxP : 1];
  __shared__ float scale[32];
  const int lane = threadIdx.x & 63;
  const int rg = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, i16 = lane & 15;
  int e, cnt;
  const int32_t *pair;
  if constexpr (SCAN) {
    for (int p = threadIdx.x; p < a.P; p += 256) ids[p] = a.ids[p];
    __syncthreads();
    if (!find_pairs(a, ids, blockIdx.y, own, lane, e, cnt)) return;
    pair = own;
  } else {
    if ((int)blockIdx.y >= uload(a.lists)) return;
    e = uload(a.lists + 1 + blockIdx.y);
    const int32_t *start = a.lists + 1 + a.E;
    const int p0 = uload(start + e);
    cnt = uload(start + e + 1) - p0;
    pair = start + a.E + 1 + p0;
  }
  const int t0 = blockIdx.x * TR, rows = min(TR, (a.H >> 6) - t0);
  const RowMeta meta(a.dn, e * (a.H >> 6) + t0);
  const int c1 = rows * a.dn.C;
  float *d = a.d + t0 * 64 + rg * 16 + i16;
  if constexpr (SRC != kDirect) {
    const int cstride = a.I + 16;  // rows 16 bytes apart in the banks
    auto fill = [&](int b, int n) __attribute__((always_inline)) {
      if constexpr (SRC == kQuantize) {
        for (int t = rg; t < n; t += 4) {
          const int p = pair[b + t];
          HRow hr;
          hr.load(a.h + (size_t)p * a.I, a.I, lane);
          const float sc = hr.quantize(a.I, codes + (size_t)t * cstride, lane);
          if (lane == 0) scale[t] = sc * a.weights[p];
        }
      } else {
        const int n16 = a.I >> 4;  // 16-byte pieces of a row
        for (int o = threadIdx.x; o < n * n16; o += 256) {
          const int t = o / n16, c = o - t * n16;
          *reinterpret_cast<v4i *>(codes + (size_t)t * cstride + 16 * c) =
              load16(a.qh + (size_t)pair[b + t] * a.I + 16 * c);
        }
        if ((int)threadIdx.x < n) {
          const int p = pair[b + threadIdx.x];
          scale[threadIdx.x] = a.sh[p] * a.weights[p];
        }
      }
      // (LDS writes done; the weights' loads stay open)
      __builtin_amdgcn_s_waitcnt(0xC07F);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };
    // rows past the last hold older codes; not stored
    auto store = [&](int b, int n, int row, int q, const float (&F)[4]) __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = 16 * q + 4 * g + k;
        if (t < n) d[(size_t)pair[b + t] * a.H + row * 64] = F[k] * scale[t];
      }
    };
    for (int b = held * blockIdx.z; b < cnt; b += held * gridDim.z) {
      const int n = min(held, cnt - b);
      const int8_t *x[2] = {codes + (size_t)i16 * cstride, codes + (size_t)(16 + i16) * cstride};
      if (n > 16) {
        DownPipe<BK, 2, true> pipe(a.dn, meta, rg, 0, c1, lane, x);
        if (b) __syncthreads();  // the last pass's codes have been read
        fill(b, n);
        pipe.run(x, [&](int row, const float (&F)[2][4]) __attribute__((always_inline)) {
          store(b, n, row, 0, F[0]);
          store(b, n, row, 1, F[1]);
        });
      } else {
        const int8_t *x1[1] = {x[0]};
        DownPipe<BK, 1, true> pipe(a.dn, meta, rg, 0, c1, lane, x1);
        if (b) __syncthreads();
        fill(b, n);
        pipe.run(x1, [&](int row, const float (&F)[1][4]) __attribute__((always_inline)) { store(b, n, row, 0, F[0]); });
      }
    }
  } else {
    for (int b = held * blockIdx.z; b < cnt; b += held * gridDim.z) {  // (held = 32)
      const int8_t *x[2];
      int pr[2][4];
      float sc[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        x[n] = a.qh + (size_t)pair[min(b + 16 * n + i16, cnt - 1)] * a.I;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          pr[n][k] = pair[min(b + 16 * n + 4 * g + k, cnt - 1)];
          sc[n][k] = a.sh[pr[n][k]] * a.weights[pr[n][k]];
        }
      }
      auto store = [&](int row, int n, const float (&F)[4]) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (b + 16 * n + 4 * g + k < cnt) d[(size_t)pr[n][k] * a.H + row * 64] = F[k] * sc[n][k];
      };
      if (cnt - b > 16) {
        DownPipe<BK, 2, false> pipe(a.dn, meta, rg, 0, c1, lane, x);
        pipe.run(x, [&](int row, const float (&F)[2][4]) __attribute__((always_inline)) {
          store(row, 0, F[0]);
          store(row, 1, F[1]);
        });
      } else {
        const int8_t *x1[1] = {x[0]};
        DownPipe<BK, 1, false> pipe(a.dn, meta, rg, 0, c1, lane, x1);
        pipe.run(x1, [&](int row, const float (&F)[1][4]) __attribute__((always_inline)) { store(row, 0, F[0]); });
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

// Workgroups side by side over an expert's passes of `pass` pairs, where experts
// are few and their tokens many: as many as the passes of an expert with the
// average number of pairs, while the waves (of one pass each) fit the chip.
// (1000 tokens, 8 experts of 2048 x 1024, top 2: down 70 us with an expert's passes
// one after another, 33 side by side; 1024 tokens at one expert of 4096 x 512:
// gate/up 300 and 38 us, down 140 and 18.)
int passes_abreast(const MoeArgs &a, int slots, int pass, long long waves) {
  const int want = (a.P + slots * pass - 1) / (slots * pass);
  const long long room = 4096 / waves;
  return (int)(room < 1 ? 1 : room < want ? room : want);
}

template <int BK, int MODE, int S>
void launch_gate_up_s(const MoeArgs &a, int slots, hipStream_t stream) {
  const int Z = MODE == kChoose ? 1 : passes_abreast(a, slots, gu_two(S) ? 32 : 16, (long long)S * slots * (a.I / 16));
  const dim3 g(a.I / 16 / (gu_waves(S) / S), slots, Z), b(gu_waves(S) * 64);
  if constexpr (MODE != kChoose) {
    hipLaunchKernelGGL((moe_gate_up_kernel<BK, MODE, 1, S>), g, b, 0, stream, a);
  } else {
    if (a.E <= 64) hipLaunchKernelGGL((moe_gate_up_kernel<BK, MODE, 1, S>), g, b, 0, stream, a);
    else if (a.E <= 128) hipLaunchKernelGGL((moe_gate_up_kernel<BK, MODE, 2, S>), g, b, 0, stream, a);
    else hipLaunchKernelGGL((moe_gate_up_kernel<BK, MODE, 4, S>), g, b, 0, stream, a);
  }
}

// Column ranges: enough waves to fill the chip (about 4096), one range where
// the experts' feature groups do by themselves.  (5 tokens, 27 experts of 2560 x
// 1280, 1600 groups: 20.4 us with 2 ranges, 19.8 with 4, which need the choice in
// a launch of its own; 32 tokens, 32 experts of 4096 x 1536: 42.4 us with one, 43.9
// with two.)
// Passes of 32 pairs over an expert with the average number count like experts,
// since they may run side by side (1000 tokens, 8 experts of 2048 x 1024: 40 us
// with the one range that this gives, 103 with the 8 for the experts alone).
int gate_up_split(const MoeArgs &a) {
  const long long slots = a.P < a.E ? a.P : a.E, passes = (a.P + 32 * slots - 1) / (32 * slots);
  const long long groups = slots * passes * (a.I / 16);
  return groups <= 512 ? 8 : groups <= 1024 ? 4 : groups <= 2048 ? 2 : 1;
}

template <int BK, int MODE>
void launch_gate_up(const MoeArgs &a, hipStream_t stream) {
  const int slots = a.P < a.E ? a.P : a.E;
  switch (gate_up_split(a)) {
    case 8: return launch_gate_up_s<BK, MODE, 8>(a, slots, stream);
    case 4: return launch_gate_up_s<BK, MODE, 4>(a, slots, stream);
    case 2: return launch_gate_up_s<BK, MODE, 2>(a, slots, stream);
    default:  // (more workgroups than a fused choice takes)
      if constexpr (MODE != kChoose) launch_gate_up_s<BK, MODE, 1>(a, slots, stream);
  }
}

// The choice is made inside gate/up where its workgroups run in one round (two
// per CU): each of them pays the choice once, which is then cheaper than the
// launch of its own.
bool fused_choice(const MoeArgs &a) {
  if (a.M > kChooseMaxM || a.E > 256 || a.rt.KS > 1) return false;
  const int S = gate_up_split(a);
  return (long long)(a.P < a.E ? a.P : a.E) * (a.I / 16) / (gu_waves(S) / S) <= 512;
}

// Consecutive tile rows per workgroup: as many as leave 4096 waves (what the
// registers hold), at most 4.  The rows of one walk follow one another without
// a pause: 200 tokens, 128 experts of 2048 x 768: 58 us with one row, 45 us
// with 4; 32 tokens, 32 experts of 4096 x 1536: 31 us with one, 27 us with 2.
int down_rows_per_group(long long waves) { return waves >= 4 * 4096 ? 4 : waves >= 2 * 4096 ? 2 : 1; }

template <int BK, int SRC, bool SCAN>
void launch_down_pairs(const MoeArgs &a, hipStream_t stream) {
  const int slots = a.P < a.E ? a.P : a.E, trows = a.H / 64;
  const int TR = down_rows_per_group(4LL * slots * trows);
  // Rows of codes in LDS: 16 where an expert has up to 4 pairs on average, so that
  // more workgroups fit (128 pairs over 32 experts of 4096 x 1536: 27.7 us with
  // 16 rows, 35.6 with 32).
  const int held = SRC != kDirect && a.P <= 4LL * a.E ? 16 : 32;
  const size_t lds = SRC == kDirect ? 0 : (size_t)held * (a.I + 16);
  if (lds > 64 * 1024 - 8 * 1024)
    (void)hipFuncSetAttribute(reinterpret_cast<const void *>(moe_down_kernel<BK, SRC, SCAN>),
                              hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  const int Z = passes_abreast(a, slots, held, 4LL * slots * ((trows + TR - 1) / TR));
  hipLaunchKernelGGL((moe_down_kernel<BK, SRC, SCAN>), dim3((trows + TR - 1) / TR, slots, Z), dim3(256), lds, stream, a,
                     TR, held);
}

template <int BK>
hipError_t launch_down(const MoeArgs &a, hipStream_t stream) {
  hipError_t e;
  if (a.P <= kRowsMaxP && a.I <= kFuseqMaxI) {
    const size_t lds = sizeof(RowsLds) + (size_t)a.P * (a.I + 16);
    hipLaunchKernelGGL(moe_down_rows_kernel<BK>, dim3(a.H / 16), dim3(1024), lds, stream, a);
    return hipGetLastError();
  }
  // The rows of an expert are quantized by each of its H / 64 workgroups where
  // they are few (8 per expert on average), else once by a launch of their own.
  // (Rows of pairs without an expert hold anything; their codes are not read.)
  const bool scan = a.P <= kScanMaxP;
  if (a.P <= 8LL * a.E && a.I <= kFuseqMaxI) {
    scan ? launch_down_pairs<BK, kQuantize, true>(a, stream) : launch_down_pairs<BK, kQuantize, false>(a, stream);
  } else {
    if ((e = launch_quant_act(a.h, a.P, a.I, a.qh, a.sh, stream)) != hipSuccess) return e;
    if (a.I <= kFuseqMaxI)
      scan ? launch_down_pairs<BK, kCopy, true>(a, stream) : launch_down_pairs<BK, kCopy, false>(a, stream);
    else
      scan ? launch_down_pairs<BK, kDirect, true>(a, stream) : launch_down_pairs<BK, kDirect, false>(a, stream);
  }
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(moe_combine_kernel, dim3((a.H / 4 + 255) / 256, a.M), dim3(256), 0, stream, a);
  return hipGetLastError();
}

// gate/up and down for ids that are there: lists only where the pairs are too
// many for every workgroup to look through.
hipError_t launch_experts(const MoeArgs &a, int bk1, int bk2, hipStream_t stream) {
  hipError_t e;
  const bool scan = a.P <= kScanMaxP;
  if (!scan) {
    hipLaunchKernelGGL(moe_lists_kernel, dim3(1), dim3(1024), 0, stream, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (bk1 == 128) scan ? launch_gate_up<128, kScan>(a, stream) : launch_gate_up<128, kLists>(a, stream);
  else scan ? launch_gate_up<64, kScan>(a, stream) : launch_gate_up<64, kLists>(a, stream);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  return bk2 == 128 ? launch_down<128>(a, stream) : launch_down<64>(a, stream);
}

MoeArgs moe_args(const MoeShape &s, const PackedView &gu, const PackedView &dn, const int8_t *qx, const float *sx,
                 int32_t *ids, float *weights, float *Y, const MoeWs &ws) {
  MoeArgs a;
  a.gu = packed_of(gu);
  a.dn = packed_of(dn);
  a.rt = RouteArgs{};
  a.qx = qx; a.sx = sx; a.ids = ids; a.weights = weights; a.lists = ws.lists;
  a.h = ws.h; a.qh = ws.qh; a.sh = ws.sh; a.d = ws.d; a.Y = Y;
  a.M = s.pass(); a.top_k = s.top_k; a.E = s.E; a.H = s.H; a.I = s.I; a.P = s.pairs();
  return a;
}

// All tokens in passes of up to 1024 (one launch sequence after another on the
// stream, so they share the workspace).
hipError_t launch_passes(const MoeShape &s, MoeArgs a, int bk1, int bk2, hipStream_t stream) {
  for (int m = 0; m < s.M; m += s.pass()) {
    a.M = min(s.pass(), s.M - m);
    a.P = a.M * s.top_k;
    const hipError_t e = launch_experts(a, bk1, bk2, stream);
    if (e != hipSuccess) return e;
    a.qx += (size_t)a.M * s.H;
    a.sx += a.M;
    a.ids += (size_t)a.M * s.top_k;
    a.weights += (size_t)a.M * s.top_k;
    a.Y += (size_t)a.M * s.H;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_moe_experts(const MoeShape &s, const PackedView &gu, const PackedView &dn, const int8_t *qx,
                              const float *sx, const int32_t *ids, const float *weights, float *Y,
                              const MoeWs &ws, hipStream_t stream) {
  // the kernels of this path only read ids and weights
  const MoeArgs a = moe_args(s, gu, dn, qx, sx, const_cast<int32_t *>(ids), const_cast<float *>(weights), Y, ws);
  return launch_passes(s, a, gu.bK, dn.bK, stream);
}

hipError_t launch_moe_layer(const MoeShape &s, const PackedView &gu, const PackedView &dn, const RouteArgs &rt,
                            int8_t *qx, float *sx, float *Y, const MoeWs &ws, hipStream_t stream) {
  MoeArgs a = moe_args(s, gu, dn, qx, sx, rt.ids, rt.weights, Y, ws);
  a.rt = rt;
  hipError_t e = launch_route_front(rt, qx, sx, stream);
  if (e != hipSuccess) return e;
  if (fused_choice(a)) {
    if (gu.bK == 128) launch_gate_up<128, kChoose>(a, stream);
    else launch_gate_up<64, kChoose>(a, stream);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    return dn.bK == 128 ? launch_down<128>(a, stream) : launch_down<64>(a, stream);
  }
  if ((e = launch_route_choice(rt, stream)) != hipSuccess) return e;
  return launch_passes(s, a, gu.bK, dn.bK, stream);
}

}  // namespace aq
