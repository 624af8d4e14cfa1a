// C-ABI entry points of a sparse layer's feed-forward half and of the answer:
// routing, the experts' products, the residual stream with its norms, log
// probabilities.  As in abi.hip, every argument is validated before anything is
// enqueued.
#include <cmath>

#include "oq_internal.h"

namespace oq {
namespace {

inline bool al(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_dtype(const char *fn, int dtype) {
  if (dtype != OQ_F32 && dtype != OQ_BF16) return fail(OQ_ERR_INVALID_ARG, "%s: type %d must be OQ_F32 or OQ_BF16", fn, dtype);
  return OQ_OK;
}

int check_router(const char *fn, const oq_router *r, int64_t T) {
  if (!r) return fail(OQ_ERR_INVALID_ARG, "%s: the router is NULL", fn);
  if (T < 0) return fail(OQ_ERR_INVALID_ARG, "%s: T < 0", fn);
  if (r->experts < 1 || r->k < 1) return fail(OQ_ERR_INVALID_ARG, "%s: experts=%d, k=%d", fn, r->experts, r->k);
  if (r->experts > 1024 || r->k > 32)
    return fail(OQ_ERR_UNSUPPORTED, "%s: experts=%d exceeds 1024 or k=%d exceeds 32", fn, r->experts, r->k);
  if (r->score != OQ_SCORE_SOFTMAX && r->score != OQ_SCORE_SIGMOID)
    return fail(OQ_ERR_INVALID_ARG, "%s: score=%d", fn, r->score);
  if (r->groups < 1 || r->groups > 64 || r->experts % r->groups)
    return fail(r->groups > 64 ? OQ_ERR_UNSUPPORTED : OQ_ERR_INVALID_ARG, "%s: %d groups of %d experts", fn, r->groups, r->experts);
  if (r->groups > 1 && r->experts > 512) return fail(OQ_ERR_UNSUPPORTED, "%s: groups of more than 512 experts", fn);
  const int each = r->experts / r->groups;
  if (r->top_groups < 1 || r->top_groups > r->groups)
    return fail(OQ_ERR_INVALID_ARG, "%s: top_groups=%d of %d", fn, r->top_groups, r->groups);
  if (r->group_best < 1 || r->group_best > 2 || (r->groups > 1 && r->group_best > each))
    return fail(OQ_ERR_INVALID_ARG, "%s: group_best=%d of groups of %d", fn, r->group_best, each);
  if (r->k > r->top_groups * each)
    return fail(OQ_ERR_INVALID_ARG, "%s: k=%d of %d open experts", fn, r->k, r->top_groups * each);
  if (!std::isfinite(r->factor)) return fail(OQ_ERR_INVALID_ARG, "%s: factor is not finite", fn);
  if (!al(r->bias, 4)) return fail(OQ_ERR_ALIGNMENT, "%s: bias misaligned", fn);
  if (T > ((int64_t)1 << 28) / r->k) return fail(OQ_ERR_UNSUPPORTED, "%s: more than 2^28 entries", fn);
  return OQ_OK;
}

int check_norm(const char *fn, const char *name, const oq_norm *n) {
  if (!n) return OQ_OK;
  if (n->kind != OQ_NORM_RMS && n->kind != OQ_NORM_LAYER) return fail(OQ_ERR_INVALID_ARG, "%s: kind %d of %s", fn, n->kind, name);
  if (!(n->eps >= 0.f) || !std::isfinite(n->eps)) return fail(OQ_ERR_INVALID_ARG, "%s: eps of %s must be finite and >= 0", fn, name);
  if (!al(n->w, 4) || !al(n->b, 4)) return fail(OQ_ERR_ALIGNMENT, "%s: vectors of %s misaligned", fn, name);
  return OQ_OK;
}

// Rows of `bytes`-byte elements, d wide: each starts 16-byte aligned.
int check_rows(const char *fn, const char *name, const void *x, int64_t ld, int64_t rows, int d, int bytes) {
  if (ld < 0 || (rows > 1 && ld < d)) return fail(OQ_ERR_INVALID_ARG, "%s: stride %lld of %s is less than %d", fn, (long long)ld, name, d);
  if (ld > INT64_MAX / 4 / (rows > 0 ? rows : 1)) return fail(OQ_ERR_UNSUPPORTED, "%s: stride %lld of %s", fn, (long long)ld, name);
  if (!al(x, 16) || (rows > 1 && ld % (16 / bytes))) return fail(OQ_ERR_ALIGNMENT, "%s: rows of %s must start 16-byte aligned", fn, name);
  return OQ_OK;
}

int check_logprobs(const char *fn, int64_t T, int32_t V, int32_t n, int32_t top) {
  if (T < 0 || V < 1 || n < 0 || top < 0) return fail(OQ_ERR_INVALID_ARG, "%s: T=%lld, V=%d, n=%d, top=%d", fn, (long long)T, V, n, top);
  if (V > (1 << 21) || n > 64 || top > 32)
    return fail(OQ_ERR_UNSUPPORTED, "%s: V=%d exceeds 2^21, n=%d exceeds 64 or top=%d exceeds 32", fn, V, n, top);
  if (top > V) return fail(OQ_ERR_INVALID_ARG, "%s: top=%d of %d", fn, top, V);
  if (T > ((int64_t)1 << 24)) return fail(OQ_ERR_UNSUPPORTED, "%s: T=%lld exceeds 2^24", fn, (long long)T);
  return OQ_OK;
}

}  // namespace
}  // namespace oq

using namespace oq;

extern "C" {

size_t oq_route_ws_bytes(int64_t T, const oq_router *r) {
  if (check_router("oq_route_ws_bytes", r, T)) return 0;
  return route_ws(T, *r);
}

int oq_route(const void *logits, int dtype, int64_t ld, int64_t T, const uint8_t *mask, const oq_router *r, int32_t *ids,
             float *weights, int32_t *offsets, int32_t *order, void *ws, size_t ws_bytes, hipStream_t stream) {
  const char *fn = "oq_route";
  int rc = check_router(fn, r, T);
  if (!rc) rc = check_dtype(fn, dtype);
  if (rc) return rc;
  const int es = dtype == OQ_F32 ? 4 : 2;
  if ((offsets == nullptr) != (order == nullptr) && !(T == 0 && offsets))
    return fail(OQ_ERR_INVALID_ARG, "%s: offsets and order must be given together", fn);
  if (T > 0 && (!logits || !ids || !weights)) return fail(OQ_ERR_INVALID_ARG, "%s: NULL operand", fn);
  if (T > 1 && ld < r->experts) return fail(OQ_ERR_INVALID_ARG, "%s: ld=%lld < %d experts", fn, (long long)ld, r->experts);
  if (ld > INT64_MAX / 4 / (T > 0 ? T : 1)) return fail(OQ_ERR_UNSUPPORTED, "%s: ld=%lld", fn, (long long)ld);
  if (!al(logits, es) || !al(ids, 4) || !al(weights, 4) || !al(offsets, 4) || !al(order, 4) || !al(ws, 16))
    return fail(OQ_ERR_ALIGNMENT, "%s: misaligned", fn);
  set_error("%s", "");
  if (T == 0 && !offsets) return OQ_OK;
  const size_t need = offsets ? route_ws(T, *r) : 0;
  if (need && (!ws || ws_bytes < need))
    return fail(OQ_ERR_WORKSPACE, "%s: workspace of %zu bytes required (got %zu)", fn, need, ws ? ws_bytes : (size_t)0);
  const RouteArgs a{logits, ld, T, mask, *r, ids, weights, offsets, order};
  return hip_status(launch_route(a, dtype == OQ_BF16, ws, stream), fn);
}

int oq_gemm_w8a8_experts(const int8_t *qa, int64_t lda, const float *a_scale, int64_t rows, int32_t K, const int8_t *w,
                         int64_t ldw, int64_t w_stride, const float *w_scale, int32_t N, int32_t E,
                         const int32_t *offsets, const int32_t *order, int64_t n, int32_t per, int act,
                         const float *mean, const float *w1, const float *bias, uint16_t *y, int64_t ldy,
                         hipStream_t stream) {
  const char *fn = "oq_gemm_w8a8_experts";
  if (rows < 0 || n < 0 || N < 0 || E < 1 || per < 1)
    return fail(OQ_ERR_INVALID_ARG, "%s: rows=%lld, n=%lld, N=%d, E=%d, per=%d", fn, (long long)rows, (long long)n, N, E, per);
  if (act != OQ_ACT_NONE && act != OQ_ACT_SWIGLU) return fail(OQ_ERR_INVALID_ARG, "%s: act=%d", fn, act);
  if (act == OQ_ACT_SWIGLU && N % 2) return fail(OQ_ERR_INVALID_ARG, "%s: N=%d must be even for OQ_ACT_SWIGLU", fn, N);
  if (K < 16 || K % 16 || K > 131056)
    return fail(OQ_ERR_UNSUPPORTED, "%s: K=%d must be a multiple of 16 in [16, 131056]", fn, K);
  if (E > 1024 || N > (1 << 20)) return fail(OQ_ERR_UNSUPPORTED, "%s: E=%d exceeds 1024 or N=%d exceeds 2^20", fn, E, N);
  if ((mean == nullptr) != (w1 == nullptr)) return fail(OQ_ERR_INVALID_ARG, "%s: mean and w1 must be given together", fn);
  if (n == 0 || N == 0) return OQ_OK;
  if (n > ((int64_t)1 << 28)) return fail(OQ_ERR_UNSUPPORTED, "%s: n=%lld exceeds 2^28", fn, (long long)n);
  if (rows < (n + per - 1) / per)
    return fail(OQ_ERR_INVALID_ARG, "%s: %lld activation rows for %lld entries, %d a row", fn, (long long)rows, (long long)n, per);
  if (!qa || !a_scale || !w || !w_scale || !offsets || !order || !y) return fail(OQ_ERR_INVALID_ARG, "%s: NULL operand", fn);
  if (lda < K || ldw < K) return fail(OQ_ERR_INVALID_ARG, "%s: lda=%lld or ldw=%lld < K=%d", fn, (long long)lda, (long long)ldw, K);
  if (lda > (1 << 23) || ldw > (1 << 23))
    return fail(OQ_ERR_UNSUPPORTED, "%s: lda=%lld or ldw=%lld exceeds 2^23", fn, (long long)lda, (long long)ldw);
  if (E > 1 && w_stride < N * ldw)
    return fail(OQ_ERR_INVALID_ARG, "%s: w_stride=%lld is less than an expert", fn, (long long)w_stride);
  if (w_stride > ((int64_t)1 << 50)) return fail(OQ_ERR_UNSUPPORTED, "%s: w_stride=%lld", fn, (long long)w_stride);
  const int out = act == OQ_ACT_SWIGLU ? N / 2 : N;
  if (ldy < out) return fail(OQ_ERR_INVALID_ARG, "%s: ldy=%lld < %d", fn, (long long)ldy, out);
  if (ldy > ((int64_t)1 << 30)) return fail(OQ_ERR_UNSUPPORTED, "%s: ldy=%lld exceeds 2^30", fn, (long long)ldy);
  if (!al(qa, 16) || !al(w, 16) || lda % 16 || ldw % 16 || (E > 1 && w_stride % 16))
    return fail(OQ_ERR_ALIGNMENT, "%s: rows of qa and w must start 16-byte aligned", fn);
  if (!al(y, 2) || !al(a_scale, 4) || !al(w_scale, 4) || !al(mean, 4) || !al(w1, 4) || !al(bias, 4) || !al(offsets, 4) || !al(order, 4))
    return fail(OQ_ERR_ALIGNMENT, "%s: y, a list or a float32 vector is misaligned", fn);
  set_error("%s", "");
  const ExpertArgs a{qa, lda, a_scale, K, w, ldw, E > 1 ? w_stride : 0, w_scale, N, E, offsets, order, n, per, mean, w1, bias, y, ldy};
  return hip_status(launch_gemm_experts(a, act, stream), fn);
}

int oq_residual_norm(const uint16_t *y, int64_t y_ld, int32_t k, const float *weights, float y_scale, const void *r,
                     int64_t r_ld, float r_scale, int r_type, int64_t T, int32_t d, const oq_norm *post,
                     const oq_norm *pre, const oq_mod *mod, void *r_out, int64_t ro_ld, uint16_t *h, int64_t h_ld,
                     hipStream_t stream) {
  const char *fn = "oq_residual_norm";
  int rc = check_dtype(fn, r_type);
  if (!rc) rc = check_norm(fn, "post", post);
  if (!rc) rc = check_norm(fn, "pre", pre);
  if (rc) return rc;
  if (T < 0 || k < 1) return fail(OQ_ERR_INVALID_ARG, "%s: T=%lld, k=%d", fn, (long long)T, k);
  if (d < 8 || d > 16384 || d % 8) return fail(OQ_ERR_UNSUPPORTED, "%s: d=%d must be a multiple of 8 in [8, 16384]", fn, d);
  if (k > 64 || T > 0x7fffffff / k) return fail(OQ_ERR_UNSUPPORTED, "%s: k=%d exceeds 64 or T k exceeds 2^31", fn, k);
  if (!weights && k != 1) return fail(OQ_ERR_INVALID_ARG, "%s: k=%d without weights", fn, k);
  if (!std::isfinite(y_scale) || !std::isfinite(r_scale)) return fail(OQ_ERR_INVALID_ARG, "%s: y_scale and r_scale must be finite", fn);
  if (T > 0 && !y && (post || (mod && mod->gate))) return fail(OQ_ERR_INVALID_ARG, "%s: post or gate without y", fn);
  if (T > 0 && !y && !r) return fail(OQ_ERR_INVALID_ARG, "%s: y and r are NULL", fn);
  if (T > 0 && !r_out && !h) return fail(OQ_ERR_INVALID_ARG, "%s: no output", fn);
  const int es = r_type == OQ_F32 ? 4 : 2;
  if (y) rc = check_rows(fn, "y", y, y_ld, T * k, d, 2);
  if (!rc && r) rc = check_rows(fn, "r", r, r_ld, T, d, es);
  if (!rc && r_out) rc = check_rows(fn, "r_out", r_out, ro_ld, T, d, es);
  if (!rc && h) rc = check_rows(fn, "h", h, h_ld, T, d, 2);
  if (rc) return rc;
  if (r && r == r_out && T > 1 && r_ld != ro_ld) return fail(OQ_ERR_INVALID_ARG, "%s: r_out is r with another stride", fn);
  if (!al(weights, 4)) return fail(OQ_ERR_ALIGNMENT, "%s: weights misaligned", fn);
  NormArgs a{y, y_ld, k, weights, y_scale, r, r_ld, r_scale, T, d, {}, {}, {}, r_out, ro_ld, h, h_ld};
  if (post) a.post = *post;
  if (pre) a.pre = *pre;
  if (mod && (mod->gate || mod->scale || mod->shift)) {
    if (mod->rows < 0 || (mod->rows < 1 && T > 0)) return fail(OQ_ERR_INVALID_ARG, "%s: the modulation has no rows", fn);
    if (!mod->row && mod->rows != 1 && mod->rows < T)
      return fail(OQ_ERR_INVALID_ARG, "%s: %lld tokens without rows, but %lld modulation rows", fn, (long long)T, (long long)mod->rows);
    rc = check_rows(fn, "gate", mod->gate, mod->ld, mod->rows, d, 2);
    if (!rc) rc = check_rows(fn, "scale", mod->scale, mod->ld, mod->rows, d, 2);
    if (!rc) rc = check_rows(fn, "shift", mod->shift, mod->ld, mod->rows, d, 2);
    if (rc) return rc;
    if (!al(mod->row, 4)) return fail(OQ_ERR_ALIGNMENT, "%s: modulation rows misaligned", fn);
    a.mod = *mod;
  }
  set_error("%s", "");
  if (T == 0) return OQ_OK;
  return hip_status(launch_residual_norm(a, r_type == OQ_BF16, stream), fn);
}

size_t oq_logprobs_ws_bytes(int64_t T, int32_t V, int32_t n, int32_t top) {
  if (check_logprobs("oq_logprobs_ws_bytes", T, V, n, top) || T == 0) return 0;
  return logprobs_ws(T, V, n, top);
}

int oq_logprobs(const void *logits, int dtype, int64_t ld, int64_t T, int32_t V, float scale, const int32_t *tokens,
                int32_t n, int32_t top, float *logprob, int32_t *rank, float *entropy, float *lse, int32_t *top_id,
                float *top_logprob, void *ws, size_t ws_bytes, hipStream_t stream) {
  const char *fn = "oq_logprobs";
  int rc = check_logprobs(fn, T, V, n, top);
  if (!rc) rc = check_dtype(fn, dtype);
  if (rc) return rc;
  if (!(scale > 0.f) || !std::isfinite(scale * ATTN_LOG2E))
    return fail(OQ_ERR_INVALID_ARG, "%s: scale must be positive and scale log2(e) finite", fn);
  if (T > 1 && ld < V) return fail(OQ_ERR_INVALID_ARG, "%s: ld=%lld < V=%d", fn, (long long)ld, V);
  if (ld > INT64_MAX / 4 / (T > 0 ? T : 1)) return fail(OQ_ERR_UNSUPPORTED, "%s: ld=%lld", fn, (long long)ld);
  if (T > 0 && !logits) return fail(OQ_ERR_INVALID_ARG, "%s: logits is NULL", fn);
  if (T > 0 && n > 0 && (!tokens || !logprob || !rank))
    return fail(OQ_ERR_INVALID_ARG, "%s: tokens, logprob or rank is NULL", fn);
  if (T > 0 && top > 0 && (!top_id || !top_logprob)) return fail(OQ_ERR_INVALID_ARG, "%s: top_id or top_logprob is NULL", fn);
  if (!al(logits, dtype == OQ_F32 ? 4 : 2) || !al(tokens, 4) || !al(logprob, 4) || !al(rank, 4) || !al(entropy, 4) || !al(lse, 4) ||
      !al(top_id, 4) || !al(top_logprob, 4) || !al(ws, 16))
    return fail(OQ_ERR_ALIGNMENT, "%s: misaligned", fn);
  set_error("%s", "");
  if (T == 0) return OQ_OK;
  const size_t need = logprobs_ws(T, V, n, top);
  if (need && (!ws || ws_bytes < need))
    return fail(OQ_ERR_WORKSPACE, "%s: workspace of %zu bytes required (got %zu)", fn, need, ws ? ws_bytes : (size_t)0);
  const LogprobArgs a{logits, ld, T, V, scale, tokens, n, top, logprob, rank, entropy, lse, top_id, top_logprob};
  return hip_status(launch_logprobs(a, dtype == OQ_BF16, ws, stream), fn);
}

}  // extern "C"
