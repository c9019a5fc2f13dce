// Host side of a decoder layer's steps between its projections (include/aq.h):
// norm and gate into INT8 rows, rotary positions, the 4-bit cache and attention
// over it.  As in aq_api.cpp every argument is checked before any HIP call.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/aq.h"
#include "aq_check.h"
#include "aq_internal.h"
#include "aq_layer.h"

namespace {

using aq::aligned16;
using aq::aligned4;

constexpr int kMaxRows = 1 << 20;
constexpr int64_t kMaxStride = 1 << 22;

bool aligned8(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
aq_status status_of(hipError_t e) { return e == hipSuccess ? AQ_OK : AQ_ERR_HIP; }
bool known_type(int t) { return t == AQ_TYPE_F32 || t == AQ_TYPE_BF16 || t == AQ_TYPE_F16; }

// Whether [a, a + na) and [b, b + nb) share a byte.
bool meet(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}
size_t span(int M, int64_t ld, int64_t n) { return 4 * ((size_t)(M - 1) * (size_t)ld + (size_t)n); }

aq_status check_cache(const aq_kv4 *c, aq::Kv4View *v) {
  if (!c) return AQ_ERR_NULL;
  int shift = 4;
  while (shift <= 8 && (1 << shift) != c->tokens) ++shift;
  if (shift > 8 || c->pages < 1 || c->heads < 1 || c->heads > 1024) return AQ_ERR_SHAPE;
  if (c->D != 64 && c->D != 128) return AQ_ERR_SHAPE;
  if (!c->codes || !c->words) return AQ_ERR_NULL;
  if (!aligned16(c->codes) || !aligned16(c->words)) return AQ_ERR_ALIGN;
  *v = aq::Kv4View{c->codes, c->words, c->pages, shift, c->heads, c->D};
  return AQ_OK;
}

// Rows of a projection's output: `n` values at a stride of ld.
aq_status check_rows(int64_t ld, int64_t n) {
  return ld < n || ld > kMaxStride || ld % 4 ? AQ_ERR_SHAPE : AQ_OK;
}

aq_status check_attn(const aq_kv4 *cache, int M, int B, int Hq, int width, aq::Kv4View *v) {
  const aq_status st = check_cache(cache, v);
  if (st != AQ_OK) return st;
  if (M < 0 || M > kMaxRows || B < (M > 0 ? 1 : 0) || B > kMaxRows) return AQ_ERR_SHAPE;
  if (Hq < 1 || Hq > 8192 || Hq % v->heads || (long long)M * Hq > (1LL << 30)) return AQ_ERR_SHAPE;
  if (width < 1 || ((long long)width << v->shift) > (1LL << 30)) return AQ_ERR_SHAPE;
  // a launch has less than 2^32 threads, 256 for each item and head: items are at most
  // M * G / 16 + 2 B tiles, where those of single tokens are B * G / 16 + B, and kItems / heads + 1
  const long long most = M > B ? M : B;
  if (most * Hq / 16 + 2LL * B * v->heads > (1LL << 24) - 2048) return AQ_ERR_SHAPE;
  return AQ_OK;
}

}  // namespace

namespace aq {

namespace {
// Tiles of p.rows rows, at most `tiles` and about `likely` of them, and how their keys are shared.  The host knows no
// length: the table's width stands for the longest.
void share(AttnPlan &p, const Kv4View &c, int B, long long tiles, long long likely, int width, bool single) {
  p.tiles = (int)tiles;
  const bool rows = p.rows <= 16;
  const int unit = rows ? 256 : 8192 / c.D;
  const long long units = (((long long)width << c.shift) + unit - 1) / unit, have = tiles * c.heads;
  // (single tokens that are not cut need no search)
  p.searched = !single || (B <= kSearched && units > 2);
  long long s = units;
  if (p.searched) {
    // as many ranges as share the keys among kItems workgroups
    if (s > kMaxRanges) s = kMaxRanges;
    // One for prompts whose tiles are that many, unless a sequence may be far longer than others (32/8 heads of
    // 128, us cut | whole: a prompt of 2048 120 | 109, of 3000 178 | 164, 8 of 250 tokens 55 | 42), and for few rows
    // over two units (the join is 4 us).
    const long long full = likely * c.heads;
    if (rows ? units <= 2 : full >= 2 * kItems || (full >= kItems && (B == 1 || units <= 64))) s = 1;
    p.splits = s < 1 ? 1 : (int)s;
    const long long shared = tiles + (kItems + c.heads - 1) / c.heads;
    p.items = (int)(tiles * p.splits < shared ? tiles * p.splits : shared);
  } else {
    // by number: some of them are launched in vain where contexts are short
    s = (s + kLongRange - 1) / kLongRange;
    if (s > 8192 / have) s = 8192 / have;
    p.splits = s < 1 ? 1 : s > kMaxRanges ? kMaxRanges : (int)s;
    p.items = (int)(tiles * p.splits);
  }
  p.index_bytes = !single && B > kSearched ? (size_t)4 * (kIndexHead + 2 * (size_t)B) : 0;
  p.part_bytes = p.splits > 1 ? (size_t)4 * p.items * c.heads * p.rows * (c.D + 4) : 0;
}
}  // namespace

AttnPlan plan_attn(const Kv4View &c, int M, int B, int Hq, int width, bool single, AttnPlan *few) {
  AttnPlan p{};
  *few = AttnPlan{};
  const int G = Hq / c.heads;
  const long long all = (long long)M * G;
  // (By the rows of all: a prompt among enough single tokens stays in tiles of few rows with them.  127 tokens over 1000 and a
  // chunk of 800 over 1000 take 174 us in one call, 49 and 55 in one each.)
  // Few rows a sequence, or few in all: tiles of 16 rows, which read the keys for each tile but leave more
  // workgroups to share them.  us by 16 rows | by 128, 8 key/value heads of 128: 64 sequences of 1000 tokens, 32 rows
  // each 68 | 73, 64 rows 121 | 89; one of 8000, 128 rows 29 | 52, 256 rows 46 | 50, 512 rows 78 | 63; one of 30000, 128
  // rows 67 | 76, 256 rows 123 | 95; 2 heads, one of 8000, 1024 rows 46 | 52, 2048 rows 78 | 64.
  const bool rows = single || all <= 32LL * B || (long long)M * Hq <= 2048;
  // Tiles of as few rows as a sequence has on average (the host knows no sequence's own), since their scores share lanes:
  // 64 tokens given with offsets, 4 rows each over 4000 keys, take 80 us in tiles of 16 rows and 54 of 4, 2 x 4 rows each
  // 79 of 16 and 63 of 8.
  p.rows = !rows ? kAttnTileRows : all <= 4LL * B ? 4 : all <= 8LL * B ? 8 : 16;
  p.upto = 1 << 30;
  if (!rows && B >= kMixed) {
    // single tokens, and what else fits their tile
    few->rows = G <= 4 ? 4 : G <= 8 ? 8 : 16;
    few->upto = p.above = G > few->rows ? G : few->rows;
    const long long tiles = (long long)B * ((few->upto + few->rows - 1) / few->rows);
    share(*few, c, B, tiles, tiles, width, false);
  }
  const long long tiles = single ? (long long)B * ((G + p.rows - 1) / p.rows) : all / p.rows + B;
  share(p, c, B, tiles, few->tiles ? all / p.rows : tiles, width, single);
  return p;
}

}  // namespace aq

namespace {
// Workspace of a call: the sums of one launch's ranges (a launch for few rows is joined before the next), then the index.
size_t sums_of(const aq::AttnPlan &p, const aq::AttnPlan &few) { return p.part_bytes > few.part_bytes ? p.part_bytes : few.part_bytes; }
size_t need(const aq::Kv4View &c, int M, int B, int Hq, int width, bool single) {
  aq::AttnPlan few;
  const aq::AttnPlan p = aq::plan_attn(c, M, B, Hq, width, single, &few);
  return sums_of(p, few) + p.index_bytes;
}
}  // namespace

extern "C" {

aq_status aq_norm_quant(const void *X, const void *R, int type, int M, int H, const void *W, int w_type,
                        double eps, void *Hout, float *Y, int8_t *qx, float *sx, void *stream) {
  if (M < 0 || M > kMaxRows || H < 64 || H % 64 || H > aq::kRowMax) return AQ_ERR_SHAPE;
  if (!known_type(type) || !known_type(w_type) || !isfinite(eps) || eps < 0) return AQ_ERR_ARG;
  if (M == 0) return AQ_OK;
  if (!X || !W || !qx || !sx) return AQ_ERR_NULL;
  if (!aligned16(X) || !aligned16(W) || !aligned16(qx) || !aligned4(sx) || !aligned16(R) || !aligned16(Hout) || !aligned16(Y))
    return AQ_ERR_ALIGN;
  const size_t n = (size_t)M * H, b = type == AQ_TYPE_F32 ? 4 : 2;
  if (Hout && ((Hout != X && meet(Hout, n * b, X, n * b)) || (R && Hout != R && meet(Hout, n * b, R, n * b)))) return AQ_ERR_ARG;
  const aq::NormArgs a{X, R, W, Hout, Y, qx, sx, M, H, type, w_type, eps};
  return status_of(aq::launch_norm_quant(a, static_cast<hipStream_t>(stream)));
}

aq_status aq_swiglu_quant(const float *GU, int64_t ld, int M, int I, float *Y, int8_t *qx, float *sx, void *stream) {
  if (M < 0 || M > kMaxRows || I < 64 || I % 64 || I > aq::kRowMax) return AQ_ERR_SHAPE;
  const aq_status st = check_rows(ld, 2 * (int64_t)I);
  if (st != AQ_OK || M == 0) return st;
  if (!GU || !qx || !sx) return AQ_ERR_NULL;
  if (!aligned16(GU) || !aligned16(qx) || !aligned4(sx) || !aligned16(Y)) return AQ_ERR_ALIGN;
  const aq::SwigluArgs a{GU, (long long)ld, Y, qx, sx, M, I};
  return status_of(aq::launch_swiglu_quant(a, static_cast<hipStream_t>(stream)));
}

aq_status aq_rope_kv4(const float *qkv, int64_t ldqkv, int M, int Hq, const aq_rope *rope, const int32_t *pos,
                      const aq_kv4 *cache, const int64_t *slots, float *Q, int64_t ldq, void *stream) {
  aq::RopeArgs a{};
  aq_status st = check_cache(cache, &a.c);
  if (st != AQ_OK) return st;
  const int D = a.c.D;
  if (M < 0 || M > kMaxRows || Hq < 0 || Hq > 8192) return AQ_ERR_SHAPE;
  st = check_rows(ldqkv, (int64_t)(Hq + 2 * a.c.heads) * D);
  if (st != AQ_OK) return st;
  if (Hq > 0 && (st = check_rows(ldq, (int64_t)Hq * D)) != AQ_OK) return st;
  if (rope) {
    if (rope->axes < 1 || rope->axes > AQ_ROPE_MAX_AXES || rope->pairs < 1 || rope->pairs > D / 2) return AQ_ERR_SHAPE;
    int sum = 0;
    for (int t = 0; t < AQ_ROPE_MAX_AXES; ++t) {
      const int p = t < rope->axes ? rope->part[t] : 0;
      if (p < 0 || p > D / 2) return AQ_ERR_SHAPE;
      sum += p;
      a.end[t] = t < rope->axes ? sum : rope->pairs;
    }
    if (sum != rope->pairs) return AQ_ERR_SHAPE;
  }
  if (M == 0) return AQ_OK;
  if (!qkv || !slots || (Hq > 0 && !Q) || (rope && (!rope->freq || !pos))) return AQ_ERR_NULL;
  if (!aligned16(qkv) || !aligned8(slots) || (Hq > 0 && !aligned16(Q)) || (rope && (!aligned4(rope->freq) || !aligned4(pos))))
    return AQ_ERR_ALIGN;
  if (Hq > 0) {
    if (Q == qkv) {
      if (ldq != ldqkv && M > 1) return AQ_ERR_ARG;
    } else if (meet(qkv, span(M, ldqkv, (int64_t)(Hq + 2 * a.c.heads) * D), Q, span(M, ldq, (int64_t)Hq * D))) {
      return AQ_ERR_ARG;
    }
  }
  a.qkv = qkv;
  a.ldqkv = ldqkv;
  a.ldq = ldq;
  a.pos = pos;
  a.slots = slots;
  a.Q = Q;
  a.M = M;
  a.Hq = Hq;
  a.pairs = rope ? rope->pairs : 0;
  a.freq = rope ? rope->freq : nullptr;
  a.interleaved = rope && rope->interleaved;
  return status_of(aq::launch_rope_kv4(a, static_cast<hipStream_t>(stream)));
}

aq_status aq_kv4_read(const aq_kv4 *cache, const int64_t *slots, int M, float *K, float *V, void *stream) {
  aq::Kv4View c;
  const aq_status st = check_cache(cache, &c);
  if (st != AQ_OK) return st;
  if (M < 0 || M > kMaxRows) return AQ_ERR_SHAPE;
  if (M == 0) return AQ_OK;
  if (!slots || !K || !V) return AQ_ERR_NULL;
  if (!aligned8(slots) || !aligned16(K) || !aligned16(V)) return AQ_ERR_ALIGN;
  return status_of(aq::launch_kv4_read(c, slots, M, K, V, static_cast<hipStream_t>(stream)));
}

size_t aq_attn_kv4_workspace_bytes(const aq_kv4 *cache, int M, int B, int Hq, int width) {
  aq::Kv4View c;
  if (check_attn(cache, M, B, Hq, width, &c) != AQ_OK || M == 0) return 0;
  // the larger of the two ways to give the sequences where both are open
  const size_t n = need(c, M, B, Hq, width, false), single = M == B ? need(c, M, B, Hq, width, true) : 0;
  return n > single ? n : single;
}

aq_status aq_attn_kv4(const float *Q, int64_t ldq, int M, int Hq, const aq_kv4 *cache, const int32_t *table,
                      int width, const int32_t *kv_len, const int32_t *cu_q, int B, float scale, float *out,
                      void *ws, size_t ws_bytes, void *stream) {
  aq::AttnArgs a{};
  aq_status st = check_attn(cache, M, B, Hq, width, &a.c);
  if (st != AQ_OK) return st;
  st = check_rows(ldq, (int64_t)Hq * a.c.D);
  if (st != AQ_OK) return st;
  if (!(scale >= 0 && scale <= 0x1p127f)) return AQ_ERR_ARG;  // (scale * log2(e) is an FP32 number)
  if (!cu_q && M != B) return AQ_ERR_ARG;
  if (M == 0) return AQ_OK;
  if (!Q || !table || !kv_len || !out) return AQ_ERR_NULL;
  if (!aligned16(Q) || !aligned16(out) || !aligned4(table) || !aligned4(kv_len) || (cu_q && !aligned4(cu_q))) return AQ_ERR_ALIGN;
  if (meet(Q, span(M, ldq, (int64_t)Hq * a.c.D), out, 4 * (size_t)M * Hq * a.c.D)) return AQ_ERR_ARG;
  aq::AttnPlan few;
  const aq::AttnPlan p = aq::plan_attn(a.c, M, B, Hq, width, cu_q == nullptr, &few);
  const size_t sums = sums_of(p, few);
  st = aq::check_workspace(ws, ws_bytes, sums + p.index_bytes);
  if (st != AQ_OK) return st;
  a.q = Q;
  a.ldq = ldq;
  a.table = table;
  a.kv_len = kv_len;
  a.cu = cu_q;
  a.out = out;
  a.part = static_cast<float *>(ws);
  a.index = p.index_bytes ? reinterpret_cast<int32_t *>(static_cast<char *>(ws) + sums) : nullptr;
  a.M = M;
  a.B = B;
  a.width = width;
  a.Hq = Hq;
  a.G = Hq / a.c.heads;
  a.scale = scale * 1.44269504088896340736f;
  for (const aq::AttnPlan &l : {few, p}) {
    if (l.tiles == 0) continue;
    a.tiles = l.tiles;
    a.splits = l.splits;
    a.items = l.items;
    a.searched = l.searched;
    a.above = l.above;
    a.upto = l.upto;
    st = status_of(aq::launch_attn_kv4(a, l, static_cast<hipStream_t>(stream)));
    if (st != AQ_OK) break;
  }
  return st;
}

}  // extern "C"
