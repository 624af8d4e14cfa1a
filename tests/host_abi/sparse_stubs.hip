// Host-only stand-ins for the launchers below abi_sparse.hip, beside those of
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

hipError_t launch_route(const RouteArgs &a, bool bf16, void *, hipStream_t) { return rec(bf16 ? "route_bf16" : "route", a.ids); }
hipError_t launch_gemm_experts(const ExpertArgs &a, int act, hipStream_t) { return rec(act ? "experts_act" : "experts", a.y); }
hipError_t launch_residual_norm(const NormArgs &a, bool bf16, hipStream_t) { return rec(bf16 ? "norm_bf16" : "norm", a.h); }
hipError_t launch_logprobs(const LogprobArgs &a, bool bf16, void *, hipStream_t) { return rec(bf16 ? "logprobs_bf16" : "logprobs", a.lse); }

}  // namespace oq
