// Host side of the marked activation quantizer (include/aq.h).  As in
// aq_api.cpp every argument is checked before any HIP call.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/aq.h"
#include "aq_check.h"
#include "aq_internal.h"

extern "C" {

aq_status aq_quant_act_marked(const float *X, int M, int K, int8_t *qx, float *sx, void *stream) {
  if (M < 0 || K <= 0 || K % 64) return AQ_ERR_SHAPE;
  if (M == 0) return AQ_OK;
  if (!X || !qx || !sx) return AQ_ERR_NULL;
  if (!aq::aligned16(X) || !aq::aligned16(qx) || !aq::aligned4(sx)) return AQ_ERR_ALIGN;
  if ((long long)M * K > (1LL << 40) || M > (1 << 30)) return AQ_ERR_SHAPE;
  return aq::launch_quant_act_marked(X, M, K, qx, sx, static_cast<hipStream_t>(stream)) == hipSuccess ? AQ_OK : AQ_ERR_HIP;
}

}  // extern "C"
