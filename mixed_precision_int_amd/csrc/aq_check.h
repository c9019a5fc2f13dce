// Argument checks shared by the host files of the C ABI (host only; no HIP
// call is made).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/aq.h"
#include "aq_internal.h"

namespace aq {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Geometry accepted by the GPU kernels.
inline aq_status check_gpu_geometry(int N, int K, int bN, int bK) {
  if (bN != kTileRows || (bK != 64 && bK != 128)) return AQ_ERR_TILE;
  if (N <= 0 || K <= 0 || N % bN || K % bK) return AQ_ERR_SHAPE;
  // int32 tile counts and K-offsets inside kernels
  if ((long long)(N / bN) * (K / bK) > (1LL << 30)) return AQ_ERR_SHAPE;
  return AQ_OK;
}

inline aq_status check_packed(const aq_packed *W) {
  if (!W) return AQ_ERR_NULL;
  aq_status st = check_gpu_geometry(W->N, W->K, W->bN, W->bK);
  if (st != AQ_OK) return st;
  const long long T = (long long)(W->N / W->bN) * (W->K / W->bK);
  if (W->T4 < 0 || W->T8 < 0 || (long long)W->T4 + W->T8 != T) return AQ_ERR_MAP;
  if (!W->labels || !W->row_off4 || !W->row_off8) return AQ_ERR_NULL;
  if (!aligned4(W->labels)) return AQ_ERR_ALIGN;
  if (W->T4 > 0 && (!W->w4 || !W->s4)) return AQ_ERR_NULL;
  if (W->T8 > 0 && (!W->w8 || !W->s8)) return AQ_ERR_NULL;
  if (!aligned4(W->row_off4) || !aligned4(W->row_off8)) return AQ_ERR_ALIGN;
  if (W->meta_host && !aligned4(W->meta_host)) return AQ_ERR_ALIGN;
  if (W->T4 > 0 && (!aligned16(W->w4) || !aligned16(W->s4))) return AQ_ERR_ALIGN;
  if (W->T8 > 0 && (!aligned16(W->w8) || !aligned16(W->s8))) return AQ_ERR_ALIGN;
  return AQ_OK;
}

inline aq_status check_workspace(void *ws, size_t ws_bytes, size_t need) {
  if (need == 0) return AQ_OK;
  if (!ws || ws_bytes < need) return AQ_ERR_WORKSPACE;
  if (!aligned16(ws)) return AQ_ERR_ALIGN;
  return AQ_OK;
}

}  // namespace aq
