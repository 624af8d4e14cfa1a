// Host-only stand-ins for the launchers below abi_serve.hip, beside those of
// stubs.hip: each records that it was reached and the output it was handed.
#include "oq_internal.h"
#include "serve_stubs.h"
#include "stubs.h"

int g_cus = 256;

static hipError_t rec(const char *name, const void *out) {
  if (g_stub.launches++ == 0) g_stub.first_out = out;
  g_stub.last = name;
  g_stub.last_out = out;
  if (g_stub.fail_next) {
    g_stub.fail_next = 0;
    return hipErrorInvalidValue;
  }
  return hipSuccess;
}

namespace oq {

int device_cus() { return g_cus; }

hipError_t launch_weight_rpbh_w8(const float *, int, int, int64_t, const RotArgs &, int8_t *codes, int64_t, float *, float *,
                                 hipStream_t) {
  return rec("weight_rpbh_w8", codes);
}
hipError_t launch_gemm_w8a8(const int8_t *, int64_t, const float *, int64_t, int, const int8_t *, int64_t, const float *, int,
                            const float *, const float *, const float *, uint16_t *y, int64_t, hipStream_t) {
  return rec("gemm_w8a8", y);
}
hipError_t launch_heads(const HeadArgs &a, hipStream_t) { return rec(a.slot ? "heads_cache" : "heads", a.part[0].out); }
hipError_t launch_attn_prefix(const AttnArgs &a, void *, hipStream_t) { return rec("attn_prefix", a.o); }

}  // namespace oq
