// Internal interface of a decoder layer's steps between its projections: norm
// and gate into INT8 rows, rotary positions, the 4-bit cache and attention
// over it.  Launchers take validated arguments and return the launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/aq.h"
#include "aq_internal.h"

namespace aq {

// ---- rows
struct NormArgs {
  const void *X, *R;   // [M][H] of type; R or nullptr
  const void *W;       // [H] of w_type
  void *Hout;          // [M][H] of type or nullptr
  float *Y;            // [M][H] or nullptr
  int8_t *qx;
  float *sx;
  int M, H, type, w_type;
  double eps;
};
hipError_t launch_norm_quant(const NormArgs &a, hipStream_t stream);

struct SwigluArgs {
  const float *GU;
  long long ld;
  float *Y;
  int8_t *qx;
  float *sx;
  int M, I;
};
hipError_t launch_swiglu_quant(const SwigluArgs &a, hipStream_t stream);
constexpr int kRowMax = 32768;  // longest row: 1024 threads of 8 float4

// ---- cache
struct Kv4View {
  uint8_t *codes;
  uint32_t *words;
  int pages, shift, heads, D;  // 1 << shift tokens a page
};

struct RopeArgs {
  const float *qkv;
  long long ldqkv, ldq;
  const int32_t *pos;     // [axes][M]
  const float *freq;      // nullptr: nothing turns
  const int64_t *slots;
  float *Q;
  Kv4View c;
  int M, Hq, pairs, interleaved;
  int end[AQ_ROPE_MAX_AXES];  // pairs of axes 0 .. a, summed
};
hipError_t launch_rope_kv4(const RopeArgs &a, hipStream_t stream);
hipError_t launch_kv4_read(const Kv4View &c, const int64_t *slots, int M, float *K, float *V, hipStream_t stream);

// ---- attention
struct AttnArgs {
  const float *q;
  long long ldq;
  Kv4View c;
  const int32_t *table, *kv_len, *cu;  // cu nullptr: one row a sequence
  float *out;
  float *part;   // workspace: [item][head][row]{O[D], max, sum}; a tile's ranges lie Rows::stride items apart
  int M, B, width, Hq, G;
  float scale;   // scale * log2(e)
  int tiles;     // row tiles there may be
  int splits;    // ranges of keys that a tile may have; 1: all keys in one
  int items;     // (tile, range) items there may be
  int32_t *index;  // workspace where the sequences are indexed first, else nullptr (aq_attn.h)
  bool searched; // items in order of sequences and found among them, or by number
  int above, upto;  // of packed sequences those of more and of up to so many rows take part
};
// Rows of a (sequence, key/value head) are its tokens x the G query heads of
// the group, token by token.
constexpr int kMaxRanges = 64;   // a lane of the join each
// Long contexts are cut so that about as many workgroups share the keys, two to a CU (three run at once where few
// rows leave room), but into no more than kMaxRanges each: one sequence of 120000 tokens has 59 workgroups to a key/value
// head (27.9 us with one head, 37.6 with eight).  (The figures of this rule and the next two with q of few rows in three
// digits; four take 2 to 4% more.)  A workgroup costs some 8 us beside its keys (a chain: lengths, pages, codes, the
// waves' sums; and the join), a unit of 256 keys in its turn 3.  us with 512 | 768 | 1024, 8 heads: 64 x 4096
// tokens 74 | 88 | 79, 16 x 4096 25.2 | 24.4 | 24.2, three of up to 120000 39.6 | 44 | 42, 48 of up to 6000
// 27.2 | 26.4 | 26.4.
constexpr int kItems = 512;
// Sequences among which each workgroup looks for its place; beyond, packed ones are indexed first and
// single tokens are numbered.  32/8 heads of 128, a row each, us by search | index: 64 x 500 tokens 15 | 22, 100 x 2000
// 59 | 62, 140 x 2000 78 | 73, 200 x 2000 111 | 95, 4096 x 100 2088 | 388; without offsets by search | number: 65 of up to
// 8000 30 | 35, 100 of up to 8000 49 | 53, 100 x 2000 54 | 46, 200 of up to 8000 79 | 72, 200 x 2000 92 | 74.
constexpr int kSearched = 128;
constexpr int kIndexHead = 4;    // int32 in front of the index's two arrays
constexpr int kLongRange = 8;    // units of a range at least where it does not
constexpr int kAttnTileRows = 128;  // rows a workgroup of the kernel for prompts takes
// Packed sequences from which those of few rows are a launch of their own beside prompts: single tokens would each be
// a tile of 128 rows.  us together | apart: 63 tokens over 4000 beside a prompt of 512 227 | 95, over 1000 87 | 64, 16 over 2000 beside
// 2048 154 | 129, 100 over 500 beside 1500 in two 92 | 120; without single tokens, 16 prompts of 250 89 | 90, 64 of 40 42 | 44.
// What decides is the single tokens' keys, which the host does not know; the number stands for them.  Below it tokens over long
// contexts lose: 7 over 120000 beside a prompt of 512 take 1272 in one call, 220 + 34 in two; 15 over 8000 70, and 37 + 34; 3 over 1000 34,
// and 12 + 34.
constexpr int kMixed = 16;
struct AttnPlan {
  int rows;      // rows a tile
  int tiles;     // row tiles there may be, over all sequences
  int splits, items;
  bool searched;
  int above, upto;
  size_t part_bytes;    // ranges' sums
  size_t index_bytes;   // behind them: the sequences' index
};
// The call's launch, and in `few` that of the sequences of few rows (no tiles: all are in one).
AttnPlan plan_attn(const Kv4View &c, int M, int B, int Hq, int width, bool single, AttnPlan *few);
hipError_t launch_attn_kv4(const AttnArgs &a, const AttnPlan &p, hipStream_t stream);
hipError_t launch_attn_rows(const AttnArgs &a, int qc, hipStream_t stream);
hipError_t launch_attn_tiles(const AttnArgs &a, hipStream_t stream);

}  // namespace aq
