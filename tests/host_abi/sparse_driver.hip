// Validation driver for the sparse layer's entry points on the CPU, as
// serve_driver.hip is for the serving ones: well-formed and malformed arguments
// with the launches and codes expected, and the plans (real host code) over the
// ranges of their sizes.  Prints "<n> cases passed" and exits 0, or lists each
// failure and exits 1.
#include <climits>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "serve_stubs.h"
#include "sparse_plan.h"
#include "stubs.h"

namespace {

int g_cases = 0, g_fail = 0;

alignas(256) unsigned char g_buf[1 << 16];
float *F = reinterpret_cast<float *>(g_buf), *F1 = reinterpret_cast<float *>(g_buf + 1);
uint16_t *X = reinterpret_cast<uint16_t *>(g_buf), *X4 = reinterpret_cast<uint16_t *>(g_buf + 4);
int8_t *C = reinterpret_cast<int8_t *>(g_buf);
int32_t *I = reinterpret_cast<int32_t *>(g_buf);
constexpr size_t ALL = ~(size_t)0;

void expect(int line, const char *what, int rc, int code, int launches, const char *last) {
  ++g_cases;
  if (rc != code || g_stub.launches != launches || std::strcmp(g_stub.last, last)) {
    ++g_fail;
    std::printf("line %d: %s -> rc %d (want %d), launches %d (want %d), '%s' (want '%s'), last error '%s'\n", line, what, rc,
                code, g_stub.launches, launches, g_stub.last, last, oq_last_error());
  } else if (rc != OQ_OK && oq_last_error()[0] == 0) {
    ++g_fail;
    std::printf("line %d: %s -> rc %d with an empty error message\n", line, what, rc);
  }
  g_stub.launches = 0;
  g_stub.last = "";
  g_stub.fail_next = 0;
}

void truth(int line, const char *what, bool ok) {
  ++g_cases;
  if (!ok && ++g_fail < 50) std::printf("line %d: %s is false\n", line, what);
}

#define RUNS(call, name) expect(__LINE__, #call, (call), OQ_OK, 1, name)
#define NOTHING(call) expect(__LINE__, #call, (call), OQ_OK, 0, "")
#define REFUSED(call, code) expect(__LINE__, #call, (call), code, 0, "")
#define TRUE(cond) truth(__LINE__, #cond, (cond))

oq_router router(int experts, int k, int groups = 1, int top_groups = 1, int best = 1, const float *bias = nullptr) {
  return oq_router{bias, experts, k, OQ_SCORE_SIGMOID, groups, top_groups, best, 1, 1.f};
}

void routes() {
  auto call = [](int64_t T, oq_router r, int64_t ld, int dtype = OQ_F32, size_t bytes = ALL) {
    return oq_route(F, dtype, ld, T, nullptr, &r, I, F, I, I, g_buf, bytes, nullptr);
  };
  RUNS(call(100, router(64, 4), 64), "route");
  RUNS(call(100, router(64, 4), 64, OQ_BF16), "route_bf16");
  RUNS(call(1, router(64, 4), 0), "route");
  RUNS(call(1 << 23, router(1024, 32), 1024), "route");
  RUNS(call(100, router(512, 32, 64, 4, 2, F), 512), "route");
  REFUSED(call((1 << 23) + 1, router(1024, 32), 1024), OQ_ERR_UNSUPPORTED);
  REFUSED(call(INT64_MAX, router(1, 1), 1), OQ_ERR_UNSUPPORTED);
  REFUSED(call(100, router(64, 4), INT64_MAX), OQ_ERR_UNSUPPORTED);
  REFUSED(call(100, router(64, 4), INT64_MIN), OQ_ERR_INVALID_ARG);
  REFUSED(call(100, router(INT_MAX, INT_MAX), 64), OQ_ERR_UNSUPPORTED);
  REFUSED(call(100, router(64, 4, INT_MAX, INT_MAX, INT_MAX), 64), OQ_ERR_UNSUPPORTED);
  REFUSED(call(100, router(64, 4, 8, INT_MAX), 64), OQ_ERR_INVALID_ARG);
  REFUSED(call(100, router(64, 4), 64, OQ_F32, 0), OQ_ERR_WORKSPACE);
  const oq_router r = router(64, 4);
  RUNS(oq_route(nullptr, OQ_F32, 64, 0, nullptr, &r, nullptr, nullptr, I, nullptr, nullptr, 0, nullptr), "route");
  NOTHING(oq_route(nullptr, OQ_F32, 64, 0, nullptr, &r, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr));
  RUNS(oq_route(F, OQ_F32, 64, 100, g_buf, &r, I, F, nullptr, nullptr, nullptr, 0, nullptr), "route");
  g_stub.fail_next = 1;
  expect(__LINE__, "a launcher's error", call(100, router(64, 4), 64), OQ_ERR_HIP, 1, "route");
}

void products() {
  auto call = [](int64_t rows, int64_t n, int per, int K, int64_t lda, int64_t ldw, int64_t stride, int N, int E, int act, int64_t ldy) {
    return oq_gemm_w8a8_experts(C, lda, F, rows, K, C, ldw, stride, F, N, E, I, I, n, per, act, nullptr, nullptr, nullptr, X, ldy, nullptr);
  };
  RUNS(call(4, 16, 4, 64, 64, 64, 512, 8, 4, OQ_ACT_NONE, 8), "experts");
  RUNS(call(4, 16, 4, 64, 64, 64, 512, 8, 4, OQ_ACT_SWIGLU, 4), "experts_act");
  RUNS(call(4, 13, 4, 64, 64, 64, 512, 8, 4, OQ_ACT_NONE, 8), "experts");
  RUNS(call(4, 16, 4, 64, 64, 64, 0, 8, 1, OQ_ACT_NONE, 8), "experts");
  RUNS(call(1 << 28, 1 << 28, 1, 131056, 1 << 23, 1 << 23, (int64_t)1 << 50, 1 << 20, 1024, OQ_ACT_NONE, 1 << 30), "experts");
  RUNS(call(1, 1 << 28, INT_MAX, 16, 16, 16, 16, 1, 1024, OQ_ACT_NONE, 1), "experts");
  NOTHING(call(0, 0, 1, 64, 0, 0, 0, 8, 4, OQ_ACT_NONE, 0));
  NOTHING(call(4, 16, 4, 64, 64, 64, 512, 0, 4, OQ_ACT_NONE, 8));
  REFUSED(call(3, 16, 4, 64, 64, 64, 512, 8, 4, OQ_ACT_NONE, 8), OQ_ERR_INVALID_ARG);
  REFUSED(call(INT64_MAX, INT64_MAX, INT_MAX, 64, 64, 64, 512, 8, 4, OQ_ACT_NONE, 8), OQ_ERR_UNSUPPORTED);
  REFUSED(call(4, 16, 4, 64, 64, 64, 511, 8, 4, OQ_ACT_NONE, 8), OQ_ERR_INVALID_ARG);
  REFUSED(call(4, 16, 4, 64, 64, 64, INT64_MIN, 8, 4, OQ_ACT_NONE, 8), OQ_ERR_INVALID_ARG);
  REFUSED(call(4, 16, 4, 64, INT64_MIN, 64, 512, 8, 4, OQ_ACT_NONE, 8), OQ_ERR_INVALID_ARG);
  REFUSED(call(4, 16, 4, 64, 64, 64, 512, 8, 4, OQ_ACT_NONE, INT64_MIN), OQ_ERR_INVALID_ARG);
  REFUSED(call(4, 16, 4, 64, 64, 64, 512, INT_MAX, 4, OQ_ACT_NONE, INT64_MAX), OQ_ERR_UNSUPPORTED);
}

void norms() {
  const oq_norm rms{F, nullptr, OQ_NORM_RMS, 1e-6f}, bad{F, F1, OQ_NORM_LAYER, 0.f};
  auto call = [&](int64_t T, int k, int d, int64_t ld, int type, const oq_norm *post, const oq_mod *mod, void *r_out) {
    return oq_residual_norm(X, ld, k, F, 1.f, F, ld, 1.f, type, T, d, post, &rms, mod, r_out, ld, X, ld, nullptr);
  };
  RUNS(call(10, 2, 64, 64, OQ_BF16, &rms, nullptr, X), "norm_bf16");
  RUNS(call(10, 2, 64, 64, OQ_F32, nullptr, nullptr, X), "norm");
  RUNS(call(1, 1, 16384, 0, OQ_F32, nullptr, nullptr, nullptr), "norm");
  RUNS(call(0x7fffffff / 64, 64, 16384, 16384, OQ_BF16, nullptr, nullptr, nullptr), "norm_bf16");
  NOTHING(call(0, 2, 64, 64, OQ_BF16, &rms, nullptr, X));
  REFUSED(call(10, 2, 64, 64, OQ_BF16, &bad, nullptr, X), OQ_ERR_ALIGNMENT);
  REFUSED(call(10, 2, 64, INT64_MAX - 7, OQ_BF16, nullptr, nullptr, X), OQ_ERR_UNSUPPORTED);
  REFUSED(call(10, 2, 64, INT64_MIN, OQ_BF16, nullptr, nullptr, X), OQ_ERR_INVALID_ARG);
  REFUSED(call(INT64_MAX, 2, 64, 64, OQ_BF16, nullptr, nullptr, X), OQ_ERR_UNSUPPORTED);
  REFUSED(call(10, INT_MIN, 64, 64, OQ_BF16, nullptr, nullptr, X), OQ_ERR_INVALID_ARG);
  const oq_mod one{X, nullptr, X, nullptr, 0, 1}, many{X, X, X, I, 64, INT64_MAX / 256}, few{X, X, X, nullptr, 64, 9}, none{nullptr, nullptr, nullptr, nullptr, -5, -5},
      far{X, X, X, I, INT64_MAX, 2};
  RUNS(call(10, 2, 64, 64, OQ_BF16, nullptr, &one, X), "norm_bf16");
  RUNS(call(10, 2, 64, 64, OQ_BF16, nullptr, &many, X), "norm_bf16");
  RUNS(call(10, 2, 64, 64, OQ_BF16, nullptr, &none, X), "norm_bf16");
  REFUSED(call(10, 2, 64, 64, OQ_BF16, nullptr, &few, X), OQ_ERR_INVALID_ARG);
  REFUSED(call(10, 2, 64, 64, OQ_BF16, nullptr, &far, X), OQ_ERR_UNSUPPORTED);
  REFUSED(oq_residual_norm(X4, 64, 1, nullptr, 1.f, nullptr, 0, 1.f, OQ_BF16, 4, 64, nullptr, nullptr, nullptr, nullptr, 0, X, 64, nullptr), OQ_ERR_ALIGNMENT);
  RUNS(oq_residual_norm(X, 64, 1, nullptr, 1.f, nullptr, -9, 1.f, OQ_BF16, 4, 64, nullptr, nullptr, nullptr, nullptr, -9, X, 64, nullptr), "norm_bf16");
}

void answers() {
  auto call = [](int64_t T, int V, int64_t ld, int n, int top, int dtype, size_t bytes = ALL) {
    return oq_logprobs(F, dtype, ld, T, V, 1.f, I, n, top, F, I, F, F, I, F, g_buf, bytes, nullptr);
  };
  RUNS(call(10, 1000, 1000, 2, 5, OQ_F32), "logprobs");
  RUNS(call(10, 1000, 1001, 0, 0, OQ_BF16), "logprobs_bf16");
  RUNS(call(1 << 24, 1 << 21, 1 << 21, 64, 32, OQ_F32), "logprobs");
  NOTHING(call(0, 1000, 0, 2, 5, OQ_F32));
  REFUSED(call(10, 1000, INT64_MAX, 2, 5, OQ_F32), OQ_ERR_UNSUPPORTED);
  REFUSED(call(10, INT_MAX, INT64_MAX, 2, 5, OQ_F32), OQ_ERR_UNSUPPORTED);
  REFUSED(call(10, INT_MIN, 0, 2, 5, OQ_F32), OQ_ERR_INVALID_ARG);
  REFUSED(call(1, 1000000, 0, 2, 5, OQ_F32, oq_logprobs_ws_bytes(1, 1000000, 2, 5) - 1), OQ_ERR_WORKSPACE);
  RUNS(oq_logprobs(F, OQ_F32, 0, 1, 10, 1.f, nullptr, 0, 0, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr), "logprobs");
}

void route_plans() {
  for (int64_t T : {0ll, 1ll, 31ll, 32ll, 33ll, 1000ll, 8191ll, 32768ll, 1000003ll, 1ll << 28})
    for (int E = 1; E <= 1024; ++E)
      for (int groups = 1; groups <= 64; ++groups) {
        if (E % groups || (groups > 1 && E > 512)) continue;
        for (int open : {1, groups}) {
          const oq_router r = router(E, 1, groups, open);
          const oq::RoutePlan p = oq::route_plan(T, r);
          bool ok = p.l.c >= 1 && p.l.c <= 16 && p.l.groups * p.l.lanes <= 64 && p.l.lanes * p.l.c >= p.l.each && p.l.each * p.l.groups == E;
          ok = ok && p.plain == (open == groups);
          ok = ok && (p.solo ? p.chunks == 1 && p.tokens == T : p.tokens % oq::ROUTE_WAVES == 0 && p.chunks <= oq::ROUTE_CHUNKS);
          ok = ok && p.chunks * p.tokens >= T && (T == 0 || (p.chunks - 1) * p.tokens < T);
          ok = ok && oq_route_ws_bytes(T, &r) == (p.solo ? 0 : (size_t)p.chunks * E * 4);
          truth(__LINE__, "route plan", ok);
        }
      }
}

void logprob_plans() {
  for (int cus : {1, 64, 256, 304}) {
    g_cus = cus;
    for (int64_t T : {1ll, 2ll, 77ll, 511ll, 513ll, 2048ll, 100003ll, 1ll << 24})
      for (int V : {1, 2, 7, 8, 9, 500, 4095, 4096, 4097, 32000, 32768, 32769, 131072, 262147, (1 << 21) - 1, 1 << 21})
        for (int top : {0, 1, 32})
          for (int n : {0, 3, 64}) {
            if (top > V) continue;
            const size_t ws = oq_logprobs_ws_bytes(T, V, n, top);
            for (int bytes : {2, 4})
              for (int lead = 0; lead < 16 / bytes; ++lead) {
                const oq::LogprobPlan p = oq::logprob_plan(T, V, bytes, lead, top);
                const int ve = 16 / bytes, pieces = (V + lead + ve - 1) / ve;
                bool ok = p.parts >= 1 && p.each >= 1 && (int64_t)p.parts * p.each >= pieces && (p.parts - 1) * p.each < pieces;
                ok = ok && p.each <= 64 * p.waves * p.nv && p.nv >= 1 && p.nv <= 8 && (p.waves == 8 || ((p.waves == 16 || p.waves == 4) && p.nv == 8));
                ok = ok && (int64_t)p.parts * top * 8 <= 65536;  // the join's keys in LDS
                const oq::LogprobScratch s = oq::logprob_scratch(T, p.parts, n, top);
                ok = ok && s.bytes <= ws && s.keys % 16 == 0 && s.ranks % 16 == 0;
                ok = ok && (p.parts == 1 || (s.ranks - s.keys >= (size_t)T * p.parts * top * 8 && s.bytes - s.ranks >= (size_t)T * p.parts * n * 4));
                truth(__LINE__, "log probability plan", ok);
              }
          }
  }
  g_cus = 256;
}

}  // namespace

int main() {
  routes();
  products();
  norms();
  answers();
  route_plans();
  logprob_plans();
  if (g_fail) {
    std::printf("%d of %d cases failed\n", g_fail, g_cases);
    return 1;
  }
  std::printf("%d cases passed\n", g_cases);
  return 0;
}
