// Host side of the per-token-factor operators of include/aq.h: the router,
// the mixture-of-experts layer and the low-rank adapters.  As in aq_api.cpp
// every argument is checked before any HIP call.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/aq.h"
#include "aq_check.h"
#include "aq_internal.h"
#include "aq_routed.h"

namespace {

using aq::aligned16;
using aq::aligned4;

aq_status status_of(hipError_t e) { return e == hipSuccess ? AQ_OK : AQ_ERR_HIP; }

aq_status check_route(int M, int K, int wr_type, int E, int top_k, int score, float scale) {
  if (M < 0 || K <= 0 || K % 64) return AQ_ERR_SHAPE;
  if (E < 1 || E > AQ_MOE_MAX_EXPERTS) return AQ_ERR_SHAPE;
  if (top_k < 1 || top_k > E || top_k > AQ_MOE_MAX_TOP_K) return AQ_ERR_ARG;
  if (wr_type != AQ_TYPE_F32 && wr_type != AQ_TYPE_BF16) return AQ_ERR_ARG;
  if (score != AQ_SCORE_SOFTMAX && score != AQ_SCORE_SIGMOID) return AQ_ERR_ARG;
  if (!isfinite(scale)) return AQ_ERR_ARG;
  if (K > (1 << 22) || M > (1 << 20)) return AQ_ERR_SHAPE;  // 32-bit offsets inside a tile; launch sizes
  return AQ_OK;
}

aq_status check_route_ptrs(const float *X, const void *Wr, const float *bias, const int32_t *ids,
                           const float *weights) {
  if (!X || !Wr || !ids || !weights) return AQ_ERR_NULL;
  if (!aligned16(X) || !aligned16(Wr) || !aligned4(ids) || !aligned4(weights) || (bias && !aligned4(bias)))
    return AQ_ERR_ALIGN;
  return AQ_OK;
}

// Geometry of the layer; fills s.
aq_status check_moe(const aq_packed *gu, const aq_packed *dn, int E, int M, int top_k, aq::MoeShape *s) {
  aq_status st = aq::check_packed(gu);
  if (st != AQ_OK) return st;
  st = aq::check_packed(dn);
  if (st != AQ_OK) return st;
  if (E < 1 || E > AQ_MOE_MAX_EXPERTS) return AQ_ERR_SHAPE;
  if (top_k < 1 || top_k > AQ_MOE_MAX_TOP_K) return AQ_ERR_ARG;
  if (M < 0 || M > (1 << 20)) return AQ_ERR_SHAPE;
  const int H = gu->K, I = dn->K;
  if (H % 64 || I % 64) return AQ_ERR_SHAPE;
  if ((long long)gu->N != 2LL * E * I || (long long)dn->N != (long long)E * H) return AQ_ERR_SHAPE;
  *s = aq::MoeShape{M, top_k, E, H, I};
  return AQ_OK;
}

// aq_moe_layer's workspace: the experts' part, the router's logits, the
// quantized rows and their scales.
struct LayerWs {
  aq::MoeWs moe;
  void *route;
  int8_t *qx;
  float *sx;
  size_t bytes;
};
LayerWs layer_ws(const aq::MoeShape &s, void *base) {
  LayerWs w;
  w.moe = aq::moe_workspace(s, base);
  const uintptr_t b = reinterpret_cast<uintptr_t>(base);
  size_t o = w.moe.bytes;
  w.route = reinterpret_cast<void *>(b + o);
  o += aq::route_workspace_bytes(s.M, s.H, s.E);
  w.qx = reinterpret_cast<int8_t *>(b + o);
  o += aq::align256((size_t)s.M * s.H);
  w.sx = reinterpret_cast<float *>(b + o);
  o += aq::align256(4 * (size_t)s.M);
  w.bytes = o;
  return w;
}

aq_status check_lora(const aq_lora *ad, int M) {
  if (!ad) return AQ_ERR_NULL;
  if (ad->L < 1 || ad->L > AQ_LORA_MAX_ADAPTERS || ad->R < 8 || ad->R > 128 || ad->R % 8) return AQ_ERR_SHAPE;
  if (ad->K <= 0 || ad->K % 64 || ad->N <= 0 || ad->N % 64) return AQ_ERR_SHAPE;
  if (ad->type != AQ_TYPE_F32 && ad->type != AQ_TYPE_BF16 && ad->type != AQ_TYPE_F16) return AQ_ERR_ARG;
  if (M < 0 || M > (1 << 20) || ad->N > (1 << 20) || ad->K > (1 << 20)) return AQ_ERR_SHAPE;
  return AQ_OK;
}

}  // namespace

extern "C" {

size_t aq_moe_route_workspace_bytes(int M, int K, int E) {
  if (M <= 0 || M > (1 << 20) || K <= 0 || K % 64 || K > (1 << 22) || E < 1 || E > AQ_MOE_MAX_EXPERTS)
    return 0;
  return aq::route_workspace_bytes(M, K, E);
}

aq_status aq_moe_route(const float *X, int M, int K, const void *Wr, int wr_type, int E, const float *bias,
                       int top_k, int score, int norm, float scale, int32_t *ids, float *weights, void *ws,
                       size_t ws_bytes, void *stream) {
  aq_status st = check_route(M, K, wr_type, E, top_k, score, scale);
  if (st != AQ_OK || M == 0) return st;
  st = check_route_ptrs(X, Wr, bias, ids, weights);
  if (st != AQ_OK) return st;
  st = aq::check_workspace(ws, ws_bytes, aq::route_workspace_bytes(M, K, E));
  if (st != AQ_OK) return st;
  const aq::RouteArgs a{X, Wr, bias, static_cast<double *>(ws), ids, weights, M, K, E,
                        wr_type, top_k, score, norm != 0, scale, aq::route_splits(M, K, E)};
  return status_of(aq::launch_route(a, static_cast<hipStream_t>(stream)));
}

size_t aq_moe_workspace_bytes(const aq_packed *gate_up, const aq_packed *down, int E, int M, int top_k) {
  aq::MoeShape s;
  if (check_moe(gate_up, down, E, M, top_k, &s) != AQ_OK || M == 0) return 0;
  return layer_ws(s, nullptr).bytes;
}

aq_status aq_moe_experts(const aq_packed *gate_up, const aq_packed *down, int E, const int8_t *qx,
                         const float *sx, int M, const int32_t *ids, const float *weights, int top_k,
                         float *Y, void *ws, size_t ws_bytes, void *stream) {
  aq::MoeShape s;
  aq_status st = check_moe(gate_up, down, E, M, top_k, &s);
  if (st != AQ_OK || M == 0) return st;
  if (!qx || !sx || !ids || !weights || !Y) return AQ_ERR_NULL;
  if (!aligned16(qx) || !aligned4(sx) || !aligned4(ids) || !aligned4(weights) || !aligned16(Y)) return AQ_ERR_ALIGN;
  st = aq::check_workspace(ws, ws_bytes, layer_ws(s, nullptr).bytes);
  if (st != AQ_OK) return st;
  return status_of(aq::launch_moe_experts(s, aq::view_of(*gate_up), aq::view_of(*down), qx, sx, ids, weights, Y,
                                          layer_ws(s, ws).moe, static_cast<hipStream_t>(stream)));
}

aq_status aq_moe_layer(const aq_packed *gate_up, const aq_packed *down, int E, const float *X, int M,
                       const void *Wr, int wr_type, const float *bias, int top_k, int score, int norm,
                       float scale, int32_t *ids, float *weights, float *Y, void *ws, size_t ws_bytes,
                       void *stream) {
  aq::MoeShape s;
  aq_status st = check_moe(gate_up, down, E, M, top_k, &s);
  if (st != AQ_OK) return st;
  st = check_route(M, s.H, wr_type, E, top_k, score, scale);
  if (st != AQ_OK || M == 0) return st;
  st = check_route_ptrs(X, Wr, bias, ids, weights);
  if (st != AQ_OK) return st;
  if (!Y) return AQ_ERR_NULL;
  if (!aligned16(Y)) return AQ_ERR_ALIGN;
  st = aq::check_workspace(ws, ws_bytes, layer_ws(s, nullptr).bytes);
  if (st != AQ_OK) return st;
  const LayerWs w = layer_ws(s, ws);
  const aq::RouteArgs a{X, Wr, bias, static_cast<double *>(w.route), ids, weights, M, s.H, E,
                        wr_type, top_k, score, norm != 0, scale, aq::route_splits(M, s.H, E)};
  return status_of(aq::launch_moe_layer(s, aq::view_of(*gate_up), aq::view_of(*down), a, w.qx, w.sx, Y, w.moe,
                                        static_cast<hipStream_t>(stream)));
}

size_t aq_lora_workspace_bytes(const aq_lora *ad, int M) {
  if (check_lora(ad, M) != AQ_OK || M == 0) return 0;
  return aq::lora_workspace_bytes(M, ad->L, ad->K, ad->N, ad->R, ad->type);
}

aq_status aq_lora_add(const aq_lora *ad, const float *X, int M, const int32_t *ids, const float *Yin,
                      int64_t ldyin, float *Y, int64_t ldy, void *ws, size_t ws_bytes, void *stream) {
  aq_status st = check_lora(ad, M);
  if (st != AQ_OK || M == 0) return st;
  if (!ad->A || !ad->B || !X || !ids || !Yin || !Y) return AQ_ERR_NULL;
  if (!aligned16(ad->A) || !aligned16(ad->B) || !aligned16(X) || !aligned16(Yin) || !aligned16(Y) ||
      !aligned4(ids) || (ad->scale && !aligned4(ad->scale)) || (ad->rank && !aligned4(ad->rank)))
    return AQ_ERR_ALIGN;
  const int64_t most = 1LL << 22;  // 32-bit byte offsets inside a tile of 64 rows
  if (ldyin < ad->N || ldy < ad->N || ldyin % 4 || ldy % 4 || ldyin > most || ldy > most) return AQ_ERR_SHAPE;
  // Y is Yin itself or apart from it
  if (Y == Yin) {
    if (ldy != ldyin && M > 1) return AQ_ERR_ARG;
  } else {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(Yin), b0 = reinterpret_cast<uintptr_t>(Y);
    const uintptr_t a1 = a0 + 4 * ((uintptr_t)(M - 1) * (uintptr_t)ldyin + (uintptr_t)ad->N);
    const uintptr_t b1 = b0 + 4 * ((uintptr_t)(M - 1) * (uintptr_t)ldy + (uintptr_t)ad->N);
    if (a0 < b1 && b0 < a1) return AQ_ERR_ARG;
  }
  st = aq::check_workspace(ws, ws_bytes, aq::lora_workspace_bytes(M, ad->L, ad->K, ad->N, ad->R, ad->type));
  if (st != AQ_OK) return st;
  const size_t v_bytes = aq::lora_v_bytes(M, ad->L, ad->K, ad->N, ad->R, ad->type);
  const aq::LoraArgs a{ad->A, ad->B, ad->scale, ad->rank, X, ids, Yin, Y, static_cast<float *>(ws),
                       reinterpret_cast<int32_t *>(static_cast<char *>(ws) + v_bytes),
                       (long long)ldyin, (long long)ldy, ad->L, ad->R, ad->K, ad->N, M, ad->type,
                       aq::lora_splits(M, ad->L, ad->K, ad->N, ad->R, ad->type)};
  return status_of(aq::launch_lora(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
