// Internal interface of the per-token-factor operators: the router, the
// mixture-of-experts layer over packed experts, and the low-rank adapters.
// Launchers take validated arguments and return the launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/aq.h"
#include "aq_internal.h"

namespace aq {

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// ---- router
struct RouteArgs {
  const float *X;      // [M][K]
  const void *Wr;      // [E][K], FP32 or BF16
  const float *bias;   // [E] or nullptr
  double *logits;      // [KS][M][E] (workspace): partial sums over KS column ranges
  int32_t *ids;        // [M][top_k]
  float *weights;      // [M][top_k]
  int M, K, E, wr_type, top_k, score, norm;
  float scale;
  int KS;
};
// Column ranges of the logits.  Up to 2048 (token, expert) pairs a wave forms
// one logit each (one range); more take 32 x 32 tiles, whose columns are cut
// until about 1280 workgroups run, five per CU, at most 16 ranges of at least
// 128 columns (1024 x 5120 x 160, logits + choice: 34.9 + 7.0 us, against 39.2 +
// 6.2 with 768 and 36.5 + 6.6 with 1536).
inline bool route_by_rows(int M, int E) { return (long long)M * E <= 2048; }
inline int route_splits(int M, int K, int E) {
  if (route_by_rows(M, E)) return 1;
  const long long tiles = (long long)((M + 31) / 32) * ((E + 31) / 32);
  long long ks = 1280 / tiles;
  if (ks > K / 128) ks = K / 128;
  return ks < 1 ? 1 : ks > 16 ? 16 : (int)ks;
}
inline size_t route_workspace_bytes(int M, int K, int E) {
  return align256((size_t)8 * route_splits(M, K, E) * M * E);
}
hipError_t launch_route(const RouteArgs &a, hipStream_t stream);  // logits, then choice
hipError_t launch_route_choice(const RouteArgs &a, hipStream_t stream);
// The logits and the per-token INT8 rows of X, one launch for few tokens.
hipError_t launch_route_front(const RouteArgs &a, int8_t *qx, float *sx, hipStream_t stream);

// ---- experts
// Geometry of a layer of E experts whose gate/up and down projections are
// packed as one projection each: expert e owns rows e*2I .. of gate_up (I
// gate rows, then I up rows) and rows e*H .. of down.
struct MoeShape {
  int M, top_k, E, H, I;
  // The experts' part takes up to 1024 tokens at a time, which bounds the
  // workspace ([pairs][I] and [pairs][H] in FP32) and what one workgroup groups
  // by expert; longer batches pass over the weights once per 1024 tokens.
  int pass() const { return M < 1024 ? M : 1024; }
  int pairs() const { return pass() * top_k; }
};
// Workspace of the experts' part (one pass).
struct MoeWs {
  int32_t *lists;  // [0] = number of active experts, then active [E], start [E + 1], pair [P]
  float *h;        // [P][I] SwiGLU output
  int8_t *qh;      // [P][I] its INT8 codes
  float *sh;       // [P] their scales
  float *d;        // [P][H] the pairs' weighted outputs
  size_t bytes;
};
inline MoeWs moe_workspace(const MoeShape &s, void *base) {
  MoeWs w;
  char *b = static_cast<char *>(base);
  const size_t P = (size_t)s.pairs();
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return reinterpret_cast<void *>(reinterpret_cast<uintptr_t>(b) + at);
  };
  w.lists = static_cast<int32_t *>(take(4 * (2 + 2 * (size_t)s.E + P)));
  w.h = static_cast<float *>(take(4 * P * s.I));
  w.qh = static_cast<int8_t *>(take(P * s.I));
  w.sh = static_cast<float *>(take(4 * P));
  w.d = static_cast<float *>(take(4 * P * s.H));
  w.bytes = o;
  return w;
}
hipError_t launch_moe_experts(const MoeShape &s, const PackedView &gu, const PackedView &dn, const int8_t *qx,
                              const float *sx, const int32_t *ids, const float *weights, float *Y,
                              const MoeWs &ws, hipStream_t stream);
// The whole layer: front, choice, experts (rt.ids and rt.weights receive the route).
hipError_t launch_moe_layer(const MoeShape &s, const PackedView &gu, const PackedView &dn, const RouteArgs &rt,
                            int8_t *qx, float *sx, float *Y, const MoeWs &ws, hipStream_t stream);

// ---- low-rank adapters
struct LoraArgs {
  const void *A, *B;     // [L][R][K], [L][N][R]
  const float *scale;    // [L] or nullptr
  const int32_t *rank;   // [L] or nullptr
  const float *X;        // [M][K]
  const int32_t *ids;    // [M]
  const float *Yin;
  float *Y;
  float *v;              // workspace: [KS][M][R] partial sums
  int32_t *lists;        // workspace: number of tiles, permuted tokens, tiles
  long long ldyin, ldy;  // row strides of Yin and Y, elements
  int L, R, K, N, M, type, KS;
};
// Tokens by rows: a wave per token and range, which reads the token's adapter
// for itself, in two launches.  Tokens in tiles of 64 of one adapter, which read
// it once: a launch more, for the lists, and three chains of load round trips.
// Rows where the bytes that they read are few, and up to half as many again where the
// pool has an adapter for every token (the ids are not known here; where the tokens
// share one of them its repeats come from the caches).  Microseconds, rows / tiles; M,
// L, R, K + N:
//   333, 8, 8, 5120 FP16 (26 MiB): 10.8 / 17.6    1000, 4, 8, 4096 BF16 (63 MiB): 14.0 / 17.8
//   40, 4, 64, 10240 FP32 (100 MiB): 16.4 / 22.4  300, 30, 16, 8192 FP32 (150 MiB): 23.2 / 17.8
//   100, 50, 64, 12288 BF16 (150 MiB): 36.0 / 27.3
// and, an adapter each, then all tokens at one:
//   64, 64, 32, 32768 BF16 (128 MiB): 32.9 / 41.4, 17.5 / 20.9
//   100, 100, 64, 12288 BF16 (150 MiB): 36.2 / 49.8, 18.4 / 24.9
//   200, 256, 32, 12288 BF16 (150 MiB): 39.2 / 49.8, 20.2 / 22.7
//   64, 64, 64, 10240 FP32 (160 MiB): 35.7 / 49.8, 13.4 / 36.8
//   48, 64, 64, 32768 BF16 (192 MiB): 44.4 / 56.8, 22.8 / 24.2
inline bool lora_by_rows(int M, int L, int K, int N, int R, int type) {
  const long long bytes = (long long)M * R * (K + N) * (type == AQ_TYPE_F32 ? 4 : 2);
  return bytes < (128LL << 20) || (M <= L && bytes <= (192LL << 20));
}
// Tiles of up to 64 tokens of one adapter (or of none): at most.
inline int lora_max_tiles(int M, int L) { return M / 64 + (L + 1 < M ? L + 1 : M); }
// Column ranges of the first launch: 512 columns (one load per adapter row) for
// rows, at most 16; for tiles about 2048 workgroups, if there are as many tiles
// as there may be, of at least 256 columns, at most 8, since each workgroup of
// the second launch reads all ranges' sums of its tokens.
inline int lora_splits(int M, int L, int K, int N, int R, int type) {
  const int nb = K / 64;
  int ks;
  if (lora_by_rows(M, L, K, N, R, type)) {
    ks = (nb + 7) / 8 < 16 ? (nb + 7) / 8 : 16;
  } else {
    ks = 2048 / lora_max_tiles(M, L) + 1;
    if (ks > nb / 4) ks = nb / 4;
    if (ks > 8) ks = 8;
  }
  return ks < 1 ? 1 : ks;
}
inline size_t lora_v_bytes(int M, int L, int K, int N, int R, int type) {
  return align256((size_t)4 * lora_splits(M, L, K, N, R, type) * M * R);
}
inline size_t lora_workspace_bytes(int M, int L, int K, int N, int R, int type) {
  return lora_v_bytes(M, L, K, N, R, type) +
         (lora_by_rows(M, L, K, N, R, type) ? 0 : align256(32 + 4 * (size_t)M + 16 * (size_t)lora_max_tiles(M, L)));
}
hipError_t launch_lora(const LoraArgs &a, hipStream_t stream);

}  // namespace aq
