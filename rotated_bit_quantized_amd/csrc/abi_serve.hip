// C-ABI entry points around the quantized linears of an attention layer: the
// 8-bit-weight product, head norm and rotary embedding, the paged cache and
// shared-prefix attention.  As in abi.hip, every argument is validated before
// anything is enqueued.
#include <cmath>

#include "oq_internal.h"

namespace oq {
namespace {

inline bool al(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Whether heads of different tokens and different numbers share elements:
// |i hs - j ld| < d for some 1 <= i < heads, 1 <= j < T.
bool heads_overlap(int64_t ld, int64_t hs, int heads, int64_t T, int d) {
  if (heads < 2 || T < 2) return false;
  if ((hs - d) / ld >= T - 1 || (ld - d) / hs >= heads - 1) return false;  // one inside the other's stride
  for (int i = 1; i < heads; ++i) {
    const __int128 at = (__int128)i * hs, j = at / ld;
    if (j >= T) break;
    if (j >= 1 && at - j * ld < d) return true;
    if (j + 1 < T && (j + 1) * ld - at < d) return true;
  }
  return false;
}

// A tensor of head vectors (T tokens, `heads` heads of d): every head must
// start 16-byte aligned, and those of an output have places of their own.
int check_heads(const char *fn, const char *name, const void *x, int64_t ld, int64_t hs, int heads, int64_t T, int d,
                bool out) {
  if (heads == 0 || T == 0) return OQ_OK;
  if (!x) return fail(OQ_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
  if (ld < 0 || hs < 0) return fail(OQ_ERR_INVALID_ARG, "%s: negative stride of %s", fn, name);
  if ((heads > 1 && hs < d) || (T > 1 && ld < d))
    return fail(OQ_ERR_INVALID_ARG, "%s: strides of %s (token %lld, head %lld) overlap heads of %d", fn, name,
                (long long)ld, (long long)hs, d);
  if (out && heads_overlap(ld, hs, heads, T, d))
    return fail(OQ_ERR_INVALID_ARG, "%s: heads of %s overlap (strides: token %lld, head %lld)", fn, name, (long long)ld,
                (long long)hs);
  if (!al(x, 16) || (T > 1 && ld % 8) || (heads > 1 && hs % 8))  // the stride over a single one is not used
    return fail(OQ_ERR_ALIGNMENT, "%s: every head of %s must start 16-byte aligned", fn, name);
  return OQ_OK;
}

int check_head_width(const char *fn, int d) {
  if (d < 8 || d > 512 || d % 8) return fail(OQ_ERR_UNSUPPORTED, "%s: head width %d must be a multiple of 8 in [8, 512]", fn, d);
  return OQ_OK;
}

int check_norm(const char *fn, float eps) {
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(OQ_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
  return OQ_OK;
}

int check_rope(const char *fn, const oq_rope *r, const int32_t *pos, int64_t T, int d) {
  if (!r) return OQ_OK;
  if (!r->cos || !r->sin) return fail(OQ_ERR_INVALID_ARG, "%s: the rotary tables are NULL", fn);
  if (!al(r->cos, 4) || !al(r->sin, 4) || !al(pos, 4)) return fail(OQ_ERR_ALIGNMENT, "%s: rotary tables misaligned", fn);
  if (r->dim < 2 || r->dim % 2 || r->dim > d)
    return fail(OQ_ERR_INVALID_ARG, "%s: rotary dim=%d must be even in [2, %d]", fn, r->dim, d);
  if (r->rows < 1) return fail(OQ_ERR_INVALID_ARG, "%s: the rotary tables have no rows", fn);
  if (!pos && T > r->rows)
    return fail(OQ_ERR_INVALID_ARG, "%s: %lld tokens without positions, but %lld table rows", fn, (long long)T, (long long)r->rows);
  return OQ_OK;
}

int check_kv(const char *fn, const oq_kv *kv) {
  if (!kv) return fail(OQ_ERR_INVALID_ARG, "%s: the cache descriptor is NULL", fn);
  if (kv->pages < 0 || kv->heads < 1 || kv->d < 1)
    return fail(OQ_ERR_INVALID_ARG, "%s: cache of %d pages, %d heads of %d", fn, kv->pages, kv->heads, kv->d);
  if (kv->page < 8 || kv->page > 1024 || (kv->page & (kv->page - 1)))
    return fail(OQ_ERR_UNSUPPORTED, "%s: page=%d must be a power of two in [8, 1024]", fn, kv->page);
  if (kv->heads > 65535) return fail(OQ_ERR_UNSUPPORTED, "%s: %d key heads", fn, kv->heads);
  if (kv->page_stride < (int64_t)kv->heads * kv->page * kv->d)
    return fail(OQ_ERR_INVALID_ARG, "%s: page_stride=%lld is less than a page", fn, (long long)kv->page_stride);
  if (kv->pages > 0 && (!kv->k || !kv->v)) return fail(OQ_ERR_INVALID_ARG, "%s: the cache is NULL", fn);
  if (!al(kv->k, 16) || !al(kv->v, 16) || kv->page_stride % 8)
    return fail(OQ_ERR_ALIGNMENT, "%s: cache pages must be 16-byte aligned", fn);
  return OQ_OK;
}

int check_attn(const char *fn, const AttnArgs &a) {
  int rc = check_kv(fn, &a.kv);
  if (rc) return rc;
  if (a.kv.d != 64 && a.kv.d != 128) return fail(OQ_ERR_UNSUPPORTED, "%s: head width %d must be 64 or 128", fn, a.kv.d);
  if (a.B < 0 || a.n_q < 1 || a.heads_q < 1)
    return fail(OQ_ERR_INVALID_ARG, "%s: B=%d, n_q=%d, heads_q=%d", fn, a.B, a.n_q, a.heads_q);
  if (a.heads_q % a.kv.heads)
    return fail(OQ_ERR_INVALID_ARG, "%s: heads_q=%d is not a multiple of %d key heads", fn, a.heads_q, a.kv.heads);
  if (a.prefix_len < 0 || a.table_ld < 0) return fail(OQ_ERR_INVALID_ARG, "%s: negative prefix_len or table_ld", fn);
  if ((int64_t)a.table_ld * a.kv.page > 0x7fffffff - 1024 || a.prefix_len > 0x7fffffff - 1024)
    return fail(OQ_ERR_UNSUPPORTED, "%s: more than 2^31 - 1024 places in one sequence", fn);
  // one product at a time: that of all three can pass 64 bits
  const int64_t most = (int64_t)1 << 30, tokens = (int64_t)a.B * a.n_q;
  if (tokens > most || tokens * a.heads_q > most)
    return fail(OQ_ERR_UNSUPPORTED, "%s: more than 2^30 query rows", fn);
  return OQ_OK;
}

}  // namespace
}  // namespace oq

using namespace oq;

extern "C" {

int oq_quant_weight_w8(const float *w, int32_t N, int32_t K, int64_t ldw, const oq_rot *rot, int8_t *codes,
                       int64_t ldc_bytes, float *scales, float *w1, hipStream_t stream) {
  const char *fn = "oq_quant_weight_w8";
  if (N < 0) return fail(OQ_ERR_INVALID_ARG, "%s: N < 0", fn);
  if (K < 16 || K > 16384 || K % 16) return fail(OQ_ERR_UNSUPPORTED, "%s: K=%d must be a multiple of 16 in [16, 16384]", fn, K);
  if (ldw < K) return fail(OQ_ERR_INVALID_ARG, "%s: ldw < K", fn);
  if (N > 0 && (!w || !codes || !scales)) return fail(OQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
  if (!al(w, 16) || ldw % 4 || !al(codes, 16) || ldc_bytes % 16) return fail(OQ_ERR_ALIGNMENT, "%s: misaligned", fn);
  RotArgs ra;
  int rc = rot_args(fn, rot, K, &ra);
  if (rc) return rc;
  if (ldc_bytes < rot_out_width(ra, K)) return fail(OQ_ERR_INVALID_ARG, "%s: ldc_bytes < %d", fn, rot_out_width(ra, K));
  set_error("%s", "");
  return hip_status(launch_weight_rpbh_w8(w, N, K, ldw, ra, codes, ldc_bytes, scales, w1, stream), fn);
}

int oq_gemm_w8a8(const int8_t *qa, int64_t lda, const float *a_scale, int64_t M, int32_t K, const int8_t *w,
                 int64_t ldw, const float *w_scale, int32_t N, const float *mean, const float *w1, const float *bias,
                 uint16_t *y, int64_t ldy, hipStream_t stream) {
  const char *fn = "oq_gemm_w8a8";
  if (M < 0 || N < 0) return fail(OQ_ERR_INVALID_ARG, "%s: negative M or N", fn);
  if (K < 16 || K % 16 || K > 131056)
    return fail(OQ_ERR_UNSUPPORTED, "%s: K=%d must be a multiple of 16 in [16, 131056]", fn, K);
  if ((mean == nullptr) != (w1 == nullptr)) return fail(OQ_ERR_INVALID_ARG, "%s: mean and w1 must be given together", fn);
  if (M == 0 || N == 0) return OQ_OK;
  if (M > ((int64_t)1 << 30)) return fail(OQ_ERR_UNSUPPORTED, "%s: M=%lld exceeds 2^30", fn, (long long)M);
  if (!qa || !a_scale || !w || !w_scale || !y) return fail(OQ_ERR_INVALID_ARG, "%s: NULL operand", fn);
  if (lda < K || ldw < K) return fail(OQ_ERR_INVALID_ARG, "%s: lda=%lld or ldw=%lld < K=%d", fn, (long long)lda, (long long)ldw, K);
  if (lda > (1 << 23) || ldw > (1 << 23))
    return fail(OQ_ERR_UNSUPPORTED, "%s: lda=%lld or ldw=%lld exceeds 2^23", fn, (long long)lda, (long long)ldw);
  if (ldy < N) return fail(OQ_ERR_INVALID_ARG, "%s: ldy=%lld < N=%d", fn, (long long)ldy, N);
  if (!al(qa, 16) || !al(w, 16) || lda % 16 || ldw % 16)
    return fail(OQ_ERR_ALIGNMENT, "%s: rows of qa and w must start 16-byte aligned", fn);
  if (!al(y, 2) || !al(a_scale, 4) || !al(w_scale, 4) || !al(mean, 4) || !al(w1, 4) || !al(bias, 4))
    return fail(OQ_ERR_ALIGNMENT, "%s: y or a float32 vector is misaligned", fn);
  set_error("%s", "");
  return hip_status(launch_gemm_w8a8(qa, lda, a_scale, M, K, w, ldw, w_scale, N, mean, w1, bias, y, ldy, stream), fn);
}

int oq_qk_norm_rope(const uint16_t *q, int64_t q_ld, int64_t q_hs, int32_t heads_q, const uint16_t *k, int64_t k_ld,
                    int64_t k_hs, int32_t heads_k, int64_t T, int32_t d, const float *w_q, const float *w_k, float eps,
                    const oq_rope *rope, const int32_t *pos, uint16_t *q_out, int64_t qo_ld, int64_t qo_hs,
                    uint16_t *k_out, int64_t ko_ld, int64_t ko_hs, hipStream_t stream) {
  const char *fn = "oq_qk_norm_rope";
  if (T < 0 || heads_q < 0 || heads_k < 0) return fail(OQ_ERR_INVALID_ARG, "%s: negative T or head count", fn);
  if (T > ((int64_t)1 << 31) - 1 || heads_q > 65535 || heads_k > 65535)
    return fail(OQ_ERR_UNSUPPORTED, "%s: T=%lld, heads %d + %d", fn, (long long)T, heads_q, heads_k);
  int rc = check_head_width(fn, d);
  if (!rc) rc = check_norm(fn, eps);
  if (!rc) rc = check_rope(fn, rope, pos, T, d);
  if (!rc) rc = check_heads(fn, "q", q, q_ld, q_hs, heads_q, T, d, false);
  if (!rc) rc = check_heads(fn, "k", k, k_ld, k_hs, heads_k, T, d, false);
  if (!rc) rc = check_heads(fn, "q_out", q_out, qo_ld, qo_hs, heads_q, T, d, true);
  if (!rc) rc = check_heads(fn, "k_out", k_out, ko_ld, ko_hs, heads_k, T, d, true);
  if (rc) return rc;
  if (!al(w_q, 4) || !al(w_k, 4)) return fail(OQ_ERR_ALIGNMENT, "%s: norm weights misaligned", fn);
  HeadArgs a;
  a.part[0] = HeadPart{q, q_ld, q_hs, heads_q, w_q, rope != nullptr, q_out, qo_ld, qo_hs};
  a.part[1] = HeadPart{k, k_ld, k_hs, heads_k, w_k, rope != nullptr, k_out, ko_ld, ko_hs};
  a.T = T;
  a.d = d;
  a.eps = eps;
  if (rope) a.rope = *rope;
  a.pos = pos;
  set_error("%s", "");
  return hip_status(launch_heads(a, stream), fn);
}

int oq_kv_append(const uint16_t *k, int64_t k_ld, int64_t k_hs, const uint16_t *v, int64_t v_ld, int64_t v_hs,
                 int64_t T, const float *w_k, float eps, const oq_rope *rope, const int32_t *pos, const int64_t *slot,
                 const oq_kv *kv, hipStream_t stream) {
  const char *fn = "oq_kv_append";
  if (T < 0) return fail(OQ_ERR_INVALID_ARG, "%s: T < 0", fn);
  if (T > ((int64_t)1 << 31) - 1) return fail(OQ_ERR_UNSUPPORTED, "%s: T=%lld", fn, (long long)T);
  int rc = check_kv(fn, kv);
  if (rc) return rc;
  const int d = kv->d;
  rc = check_head_width(fn, d);
  if (!rc) rc = check_norm(fn, eps);
  if (!rc) rc = check_rope(fn, rope, pos, T, d);
  if (!rc) rc = check_heads(fn, "k", k, k_ld, k_hs, kv->heads, T, d, false);
  if (!rc) rc = check_heads(fn, "v", v, v_ld, v_hs, kv->heads, T, d, false);
  if (rc) return rc;
  if (T > 0 && !slot) return fail(OQ_ERR_INVALID_ARG, "%s: slot is NULL", fn);
  if (!al(slot, 8) || !al(w_k, 4)) return fail(OQ_ERR_ALIGNMENT, "%s: slot or norm weights misaligned", fn);
  set_error("%s", "");
  if (kv->pages == 0) return OQ_OK;  // every slot is outside the cache
  HeadArgs a;
  a.part[0] = HeadPart{k, k_ld, k_hs, kv->heads, w_k, rope != nullptr, kv->k, 0, 0};
  a.part[1] = HeadPart{v, v_ld, v_hs, kv->heads, nullptr, false, kv->v, 0, 0};
  a.T = T;
  a.d = d;
  a.eps = eps;
  if (rope) a.rope = *rope;
  a.pos = pos;
  a.slot = slot;
  a.page_stride = kv->page_stride;
  a.slots = (int64_t)kv->pages * kv->page;
  a.page_log2 = __builtin_ctz((unsigned)kv->page);
  return hip_status(launch_heads(a, stream), fn);
}

size_t oq_attn_prefix_ws_bytes(int32_t B, int32_t n_q, int32_t heads_q, const oq_kv *kv, int32_t prefix_len,
                               int32_t table_ld) {
  if (!kv) return 0;
  AttnArgs a{};
  a.B = B;
  a.n_q = n_q;
  a.heads_q = heads_q;
  a.kv = *kv;
  a.prefix_len = prefix_len;
  a.table_ld = table_ld;
  if (check_attn("oq_attn_prefix_ws_bytes", a) || B == 0) return 0;
  return attn_prefix_ws(a);
}

int oq_attn_prefix(const uint16_t *q, int64_t q_ld, int64_t q_hs, int32_t B, int32_t n_q, int32_t heads_q,
                   const oq_kv *kv, const int32_t *prefix_table, int32_t prefix_len, const int32_t *tables,
                   int32_t table_ld, const int32_t *lens, float scale, uint16_t *o, int64_t o_ld, int64_t o_hs,
                   float *lse, void *ws, size_t ws_bytes, hipStream_t stream) {
  const char *fn = "oq_attn_prefix";
  if (!kv) return fail(OQ_ERR_INVALID_ARG, "%s: the cache descriptor is NULL", fn);
  const AttnArgs a{q, q_ld, q_hs, B, n_q, heads_q, *kv, prefix_table, prefix_len, tables, table_ld, lens, scale,
                   o, o_ld, o_hs, lse};
  int rc = check_attn(fn, a);
  if (rc) return rc;
  if (!std::isfinite(scale * ATTN_LOG2E)) return fail(OQ_ERR_INVALID_ARG, "%s: scale log2(e) is not finite", fn);
  const int64_t T = (int64_t)B * n_q;
  rc = check_heads(fn, "q", q, q_ld, q_hs, heads_q, T, kv->d, false);
  if (!rc) rc = check_heads(fn, "o", o, o_ld, o_hs, heads_q, T, kv->d, true);
  if (rc) return rc;
  if (B > 0 && prefix_len > 0 && !prefix_table) return fail(OQ_ERR_INVALID_ARG, "%s: prefix_table is NULL", fn);
  if (B > 0 && table_ld > 0 && (!tables || !lens)) return fail(OQ_ERR_INVALID_ARG, "%s: tables or lens is NULL", fn);
  if (!al(prefix_table, 4) || !al(tables, 4) || !al(lens, 4) || !al(lse, 4) || !al(ws, 16))
    return fail(OQ_ERR_ALIGNMENT, "%s: a table, lse or ws is misaligned", fn);
  set_error("%s", "");
  if (B == 0) return OQ_OK;
  const size_t need = attn_prefix_ws(a);
  if (need && (!ws || ws_bytes < need))
    return fail(OQ_ERR_WORKSPACE, "%s: workspace of %zu bytes required (got %zu)", fn, need, ws ? ws_bytes : (size_t)0);
  return hip_status(launch_attn_prefix(a, ws, stream), fn);
}

}  // extern "C"
