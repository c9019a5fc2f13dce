// The host file of a decoder layer's steps between its projections
// (aq_layer_api.cpp) with stand-in launchers, for AddressSanitizer and
// UndefinedBehaviorSanitizer: invalid calls launch nothing, valid ones launch
// once, a launch failure forced here comes back as AQ_ERR_HIP, and the plan of
// an attention call holds what its kernels assume.
#include <hip/hip_runtime_api.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include "../../mixed_precision_int_amd/csrc/aq_layer.h"

namespace {
hipError_t forced = hipSuccess;
int launches = 0;
size_t ws_bytes = 0;

#define CHECK(c)                                          \
  do {                                                    \
    if (!(c)) {                                           \
      printf("line %d: %s\n", __LINE__, #c);              \
      exit(1);                                            \
    }                                                     \
  } while (0)
}  // namespace

namespace aq {
hipError_t launch_norm_quant(const NormArgs &, hipStream_t) { return ++launches, forced; }
hipError_t launch_swiglu_quant(const SwigluArgs &, hipStream_t) { return ++launches, forced; }
hipError_t launch_rope_kv4(const RopeArgs &a, hipStream_t) {
  ++launches;
  // the axis of a pair is the number of ends at or below it, and below the last for every pair
  CHECK(a.pairs == 0 || a.end[AQ_ROPE_MAX_AXES - 1] == a.pairs);
  for (int t = 0; t + 1 < AQ_ROPE_MAX_AXES; ++t) CHECK(a.pairs == 0 || (a.end[t] >= 0 && a.end[t] <= a.end[t + 1]));
  return forced;
}
hipError_t launch_kv4_read(const Kv4View &, const int64_t *, int, float *, float *, hipStream_t) { return ++launches, forced; }
hipError_t launch_attn_kv4(const AttnArgs &a, const AttnPlan &p, hipStream_t) {
  ++launches;
  CHECK(p.splits >= 1 && p.splits <= 64 && a.splits == p.splits && a.tiles == p.tiles);  // a lane per range joins them
  const long long rows = (long long)a.M * a.G;
  // all rows, or those of sequences of few
  CHECK(a.above == 0 || a.upto == 1 << 30);
  CHECK(a.tiles >= 1 && (long long)a.tiles * p.rows >= (a.upto == 1 << 30 ? rows : (long long)(a.upto < rows ? a.upto : rows)) && (long long)a.tiles * a.c.heads <= (1LL << 30));
  CHECK(a.items == p.items && p.items >= p.tiles && (long long)p.items * a.c.heads < 1LL << 24);  // 256 threads each in 32 bits
  const size_t sums = p.splits > 1 ? (size_t)4 * p.items * a.c.heads * p.rows * (a.c.D + 4) : 0;
  CHECK(sums <= ws_bytes && (a.index != nullptr) == (a.cu && a.B > 128));
  if (a.index) {
    const size_t at = reinterpret_cast<char *>(a.index) - reinterpret_cast<char *>(a.part);
    CHECK(at % 16 == 0 && at >= sums && at + 4 * (size_t)(4 + 2 * a.B) <= ws_bytes);
  }
  return forced;
}
}  // namespace aq

int main() {
  void *fake = reinterpret_cast<void *>(uintptr_t(1) << 20);
  const float *f = static_cast<const float *>(fake);
  float *far = reinterpret_cast<float *>(uintptr_t(1) << 44);
  int8_t *q8 = reinterpret_cast<int8_t *>(far);
  const int32_t *i32 = static_cast<const int32_t *>(fake);
  const int64_t *i64 = static_cast<const int64_t *>(fake);
  for (int force = 0; force < 2; ++force) {
    forced = force ? hipErrorLaunchFailure : hipSuccess;
    const aq_status want = force ? AQ_ERR_HIP : AQ_OK;
    for (int M : {1, 255, 256, 1 << 20})
      for (int H : {64, 4096, 32768}) {
        launches = 0;
        for (int t : {AQ_TYPE_F32, AQ_TYPE_BF16, AQ_TYPE_F16})
          CHECK(aq_norm_quant(f, far, t, M, H, f, t, 1e-6, far, nullptr, q8, far, nullptr) == want);
        CHECK(aq_swiglu_quant(f, 2 * H, M, H, far, q8, far, nullptr) == want);
        CHECK(launches == 4);
        CHECK(aq_norm_quant(f, far, 0, M, H + 1, f, 0, 1e-6, far, nullptr, q8, far, nullptr) == AQ_ERR_SHAPE);
        CHECK(aq_swiglu_quant(f, H, M, H, far, q8, far, nullptr) == AQ_ERR_SHAPE);
        CHECK(launches == 4);
      }
    for (int D : {64, 128})
      for (int tokens : {16, 64, 256})
        for (int heads : {1, 8, 1024}) {
          const aq_kv4 c{7, tokens, heads, D, reinterpret_cast<uint8_t *>(far), reinterpret_cast<uint32_t *>(far)};
          launches = 0;
          for (int axes = 1; axes <= AQ_ROPE_MAX_AXES; ++axes) {
            aq_rope r{D / 2, axes & 1, axes, {0, 0, 0, 0}, f};
            for (int t = 0, left = D / 2; t < axes; ++t) left -= r.part[t] = t + 1 < axes ? left / 2 : left;
            for (int M : {1, 9, 1 << 20}) {
              const int64_t ld = (int64_t)(2 + 2 * heads) * D;
              CHECK(aq_rope_kv4(f, ld, M, 2, &r, i32, &c, i64, far, 2 * D, nullptr) == want);
              CHECK(aq_rope_kv4(far, ld, M, 2, &r, i32, &c, i64, far, ld, nullptr) == want);
              CHECK(aq_rope_kv4(f, ld, M, 2, nullptr, nullptr, &c, i64, far, 2 * D, nullptr) == want);
              CHECK(aq_rope_kv4(f, ld, M, 0, &r, i32, &c, i64, nullptr, 0, nullptr) == want);
              r.part[0] -= 1;
              CHECK(aq_rope_kv4(f, ld, M, 2, &r, i32, &c, i64, far, 2 * D, nullptr) == AQ_ERR_SHAPE);
              r.part[0] += 1;
            }
          }
          CHECK(launches == 12 * AQ_ROPE_MAX_AXES);
          launches = 0;
          CHECK(aq_kv4_read(&c, i64, 5, far, far, nullptr) == want && launches == 1);
          for (int G : {1, 4, 7, 8})
            for (int B : {1, 3, 64, 5000})
              for (int M : {1, 64, 5000, 100000})
                for (int width : {1, 40, 100000}) {
                  if ((long long)heads * G > 8192) continue;
                  const int Hq = heads * G;
                  const size_t n = aq_attn_kv4_workspace_bytes(&c, M, B, Hq, width);
                  ws_bytes = n;
                  launches = 0;
                  const bool fits = (long long)M * Hq <= (1LL << 30) && (long long)(M > B ? M : B) * Hq / 16 + 2LL * B * heads <= (1LL << 24) - 2048;
                  const aq_status w = fits ? want : AQ_ERR_SHAPE;
                  float *q = reinterpret_cast<float *>(uintptr_t(1) << 46);
                  CHECK(aq_attn_kv4(q, (int64_t)Hq * D, M, Hq, &c, i32, width, i32, i32, B, 0.1f, far, far, n, nullptr) == w);
                  if (M == B)
                    CHECK(aq_attn_kv4(q, (int64_t)Hq * D, M, Hq, &c, i32, width, i32, nullptr, B, 0.1f, far, far, n, nullptr) == w);
                  else
                    CHECK(aq_attn_kv4(q, (int64_t)Hq * D, M, Hq, &c, i32, width, i32, nullptr, B, 0.1f, far, far, n, nullptr) != AQ_OK);
                  // (a launch of its own for the sequences of few rows, which the other follows)
                  const bool two = fits && !force && (long long)M * G > 32LL * B && (long long)M * Hq > 2048 && B >= 16;
                  CHECK(launches == (fits ? M == B ? 2 : 1 : 0) + (two ? 1 : 0));
                }
        }
  }
  puts("layer host check: ok");
  return 0;
}
