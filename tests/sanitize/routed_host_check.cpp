// The host file of the per-token-factor operators (aq_routed_api.cpp) with
// stand-in launchers, for AddressSanitizer and UndefinedBehaviorSanitizer:
// invalid calls launch nothing, valid ones launch once, a launch failure
// forced here comes back as AQ_ERR_HIP, and the parts of every workspace lie
// inside the bytes that the size functions ask for, without overlap.
#include <hip/hip_runtime_api.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <vector>

#include "../../mixed_precision_int_amd/csrc/aq_routed.h"

namespace {
hipError_t forced = hipSuccess;
int launches = 0;
uintptr_t ws_base = 0, ws_end = 0;

#define CHECK(c)                                          \
  do {                                                    \
    if (!(c)) {                                           \
      printf("line %d: %s\n", __LINE__, #c);              \
      exit(1);                                            \
    }                                                     \
  } while (0)

struct Part {
  uintptr_t at, bytes;
};
void check_parts(std::vector<Part> p) {
  std::sort(p.begin(), p.end(), [](const Part &a, const Part &b) { return a.at < b.at; });
  uintptr_t end = ws_base;
  for (const Part &q : p) {
    CHECK(q.at % 16 == 0 && q.at >= end);
    end = q.at + q.bytes;
  }
  CHECK(end <= ws_end);
}
template <typename T>
Part part(const T *p, size_t n) {
  return Part{reinterpret_cast<uintptr_t>(p), n * sizeof(T)};
}
std::vector<Part> moe_parts(const aq::MoeShape &s, const aq::MoeWs &w) {
  const size_t P = (size_t)s.pairs();
  return {part(w.lists, 2 + 2 * (size_t)s.E + P), part(w.h, P * s.I), part(w.qh, P * s.I), part(w.sh, P),
          part(w.d, P * s.H)};
}
}  // namespace

namespace aq {
hipError_t launch_route(const RouteArgs &a, hipStream_t) {
  ++launches;
  CHECK(a.KS == route_splits(a.M, a.K, a.E));
  check_parts({part(a.logits, (size_t)a.KS * a.M * a.E)});
  return forced;
}
hipError_t launch_moe_experts(const MoeShape &s, const PackedView &, const PackedView &, const int8_t *, const float *,
                              const int32_t *, const float *, float *, const MoeWs &w, hipStream_t) {
  ++launches;
  check_parts(moe_parts(s, w));
  return forced;
}
hipError_t launch_moe_layer(const MoeShape &s, const PackedView &, const PackedView &, const RouteArgs &rt, int8_t *qx,
                            float *sx, float *, const MoeWs &w, hipStream_t) {
  ++launches;
  std::vector<Part> p = moe_parts(s, w);
  p.push_back(part(rt.logits, (size_t)rt.KS * rt.M * rt.E));
  p.push_back(part(qx, (size_t)s.M * s.H));
  p.push_back(part(sx, s.M));
  check_parts(p);
  return forced;
}
hipError_t launch_lora(const LoraArgs &a, hipStream_t) {
  ++launches;
  std::vector<Part> p = {part(a.v, (size_t)a.KS * a.M * a.R)};
  if (!lora_by_rows(a.M, a.L, a.K, a.N, a.R, a.type))
    p.push_back(part(a.lists, 4 + (((size_t)a.M + 3) & ~(size_t)3) + 4 * (size_t)lora_max_tiles(a.M, a.L)));
  check_parts(p);
  return forced;
}
}  // namespace aq

int main() {
  void *fake = reinterpret_cast<void *>(uintptr_t(1) << 20);
  const float *f = static_cast<const float *>(fake);
  float *Y = reinterpret_cast<float *>(uintptr_t(1) << 44);
  int32_t *ids = static_cast<int32_t *>(fake);
  void *ws = reinterpret_cast<void *>(uintptr_t(1) << 45);
  auto room = [&](size_t n) {
    ws_base = reinterpret_cast<uintptr_t>(ws);
    ws_end = ws_base + n;
    return n;
  };
  for (int M : {1, 2, 8, 9, 64, 65, 127, 1000, 1024, 1025, 5000})
    for (int E : {1, 7, 64, 130, 1024})
      for (int k : {1, 3, 32}) {
        if (k > E) continue;
        for (int force = 0; force < 2; ++force) {
          forced = force ? hipErrorLaunchFailure : hipSuccess;
          const aq_status want = force ? AQ_ERR_HIP : AQ_OK;
          const int H = 192, I = 320;
          size_t n = room(aq_moe_route_workspace_bytes(M, H, E));
          launches = 0;
          CHECK(aq_moe_route(f, M, H, fake, AQ_TYPE_BF16, E, f, k, 1, 0, 1.f, ids, Y, ws, n, nullptr) == want);
          CHECK(aq_moe_route(f, M, H, fake, AQ_TYPE_BF16, E, f, k, 1, 0, 1.f, ids, Y, ws, n - 1, nullptr) ==
                AQ_ERR_WORKSPACE);
          CHECK(aq_moe_route(f, M, H, fake, AQ_TYPE_BF16, E, f, k, 1, 0, NAN, ids, Y, ws, n, nullptr) == AQ_ERR_ARG);
          CHECK(launches == 1);
          auto packed = [&](int N, int K) {
            aq_packed p{};
            p.N = N; p.K = K; p.bN = 64; p.bK = 64;
            p.T4 = 0; p.T8 = (N / 64) * (K / 64);
            p.labels = static_cast<uint8_t *>(fake);
            p.row_off4 = p.row_off8 = ids;
            p.w8 = static_cast<int8_t *>(fake);
            p.s8 = static_cast<float *>(fake);
            return p;
          };
          const aq_packed gu = packed(E * 2 * I, H), dn = packed(E * H, I);
          n = room(aq_moe_workspace_bytes(&gu, &dn, E, M, k));
          CHECK(n > 0);
          launches = 0;
          const int8_t *qx = static_cast<const int8_t *>(fake);
          CHECK(aq_moe_experts(&gu, &dn, E, qx, f, M, ids, f, k, Y, ws, n, nullptr) == want);
          CHECK(aq_moe_layer(&gu, &dn, E, f, M, fake, 0, nullptr, k, 0, 1, 1.f, ids, Y, Y, ws, n, nullptr) == want);
          CHECK(launches == 2);
          CHECK(aq_moe_experts(&gu, nullptr, E, qx, f, M, ids, f, k, Y, ws, n, nullptr) == AQ_ERR_NULL);
          CHECK(aq_moe_experts(&gu, &gu, E, qx, f, M, ids, f, k, Y, ws, n, nullptr) == AQ_ERR_SHAPE);
          CHECK(aq_moe_layer(&gu, &dn, E, f, M, fake, 0, nullptr, E + 1, 0, 1, 1.f, ids, Y, Y, ws, n, nullptr) ==
                AQ_ERR_ARG);
          CHECK(launches == 2);
        }
      }
  for (int M : {1, 63, 64, 65, 400, 8192, 16385, 1 << 20})
    for (int L : {1, 5, 8192})
      for (int R : {8, 24, 128})
        for (int type : {AQ_TYPE_F32, AQ_TYPE_BF16, AQ_TYPE_F16})
          for (int force = 0; force < 2; ++force) {
            forced = force ? hipErrorLaunchFailure : hipSuccess;
            aq_lora ad{L, R, 64 * (1 + M % 70), 1088, type, fake, fake, nullptr, nullptr};
            const size_t n = room(aq_lora_workspace_bytes(&ad, M));
            launches = 0;
            CHECK(aq_lora_add(&ad, f, M, ids, f, 1088, Y, 1100, ws, n, nullptr) == (force ? AQ_ERR_HIP : AQ_OK));
            CHECK(aq_lora_add(&ad, f, M, ids, Y, 1100, Y, 1100, ws, n, nullptr) == (force ? AQ_ERR_HIP : AQ_OK));
            CHECK(launches == 2);
            CHECK(aq_lora_add(&ad, f, M, ids, f, 1088, Y, 1088, ws, n - 1, nullptr) == AQ_ERR_WORKSPACE);
            CHECK(aq_lora_add(&ad, f, M, ids, Y + 1088 / 2, 1088, Y, 1088, ws, n, nullptr) == AQ_ERR_ARG);
            CHECK(launches == 2);
          }
  printf("routed host check: ok\n");
  return 0;
}
