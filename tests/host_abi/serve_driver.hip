// Validation driver for the serving entry points on the CPU, as driver.hip is
// for the others: well-formed and malformed arguments with the launches and
// codes expected, and the plan of oq_attn_prefix (real host code) over the
// range of its sizes.  Prints "<n> cases passed" and exits 0, or lists each
// failure and exits 1.
#include <cmath>
#include <cstdio>
#include <cstring>

#include "attn_plan.h"
#include "serve_stubs.h"
#include "stubs.h"

namespace {

int g_cases = 0, g_fail = 0;

alignas(256) unsigned char g_buf[1 << 16];
float *F = reinterpret_cast<float *>(g_buf), *F1 = reinterpret_cast<float *>(g_buf + 1);
uint16_t *X = reinterpret_cast<uint16_t *>(g_buf), *X4 = reinterpret_cast<uint16_t *>(g_buf + 4);
int8_t *C = reinterpret_cast<int8_t *>(g_buf), *C4 = C + 4;
int32_t *I = reinterpret_cast<int32_t *>(g_buf), *I1 = reinterpret_cast<int32_t *>(g_buf + 1);
int64_t *L = reinterpret_cast<int64_t *>(g_buf), *L4 = reinterpret_cast<int64_t *>(g_buf + 4);
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

void weights() {
  auto q = [](const float *w, int N, int K, int64_t ldw, const oq_rot *rot, int8_t *c, int64_t ldc, float *s, float *w1) {
    return oq_quant_weight_w8(w, N, K, ldw, rot, c, ldc, s, w1, nullptr);
  };
  RUNS(q(F, 4, 64, 64, nullptr, C, 64, F, nullptr), "weight_rpbh_w8");
  RUNS(q(F, 4, 64, 68, nullptr, C, 80, F, F), "weight_rpbh_w8");
  oq_rot kron{OQ_ROT_KRON, 1920, 0, 0, nullptr, nullptr, nullptr};
  int32_t m, block, pad;
  TRUE(oq_kron_plan(1920, &m, &block, &pad) == OQ_OK);
  kron.rounds = m;
  kron.block = block;
  RUNS(q(F, 4, 1920, 1920, &kron, C, pad, F, nullptr), "weight_rpbh_w8");
  REFUSED(q(F, 4, 1920, 1920, &kron, C, pad - 16, F, nullptr), OQ_ERR_INVALID_ARG);
  REFUSED(q(F, -1, 64, 64, nullptr, C, 64, F, nullptr), OQ_ERR_INVALID_ARG);
  REFUSED(q(F, 4, 72, 72, nullptr, C, 80, F, nullptr), OQ_ERR_UNSUPPORTED);
  REFUSED(q(F, 4, 64, 60, nullptr, C, 64, F, nullptr), OQ_ERR_INVALID_ARG);
  REFUSED(q(nullptr, 4, 64, 64, nullptr, C, 64, F, nullptr), OQ_ERR_INVALID_ARG);
  REFUSED(q(F, 4, 64, 64, nullptr, C4, 64, F, nullptr), OQ_ERR_ALIGNMENT);
  g_stub.fail_next = 1;
  expect(__LINE__, "a launcher's error", q(F, 4, 64, 64, nullptr, C, 64, F, nullptr), OQ_ERR_HIP, 1, "weight_rpbh_w8");
}

void product() {
  auto g = [](const int8_t *qa, int64_t lda, int64_t M, int K, int64_t ldw, int N, const float *mean, const float *w1, uint16_t *y,
              int64_t ldy) { return oq_gemm_w8a8(qa, lda, F, M, K, C, ldw, F, N, mean, w1, nullptr, y, ldy, nullptr); };
  RUNS(g(C, 64, 4, 64, 64, 8, nullptr, nullptr, X, 8), "gemm_w8a8");
  RUNS(g(C, 1 << 23, 1 << 30, 131056, 1 << 23, 0x7fffffff, F, F, X, INT64_MAX), "gemm_w8a8");
  NOTHING(g(nullptr, 0, 0, 64, 0, 8, nullptr, nullptr, nullptr, 0));
  NOTHING(g(nullptr, 0, 8, 64, 0, 0, nullptr, nullptr, nullptr, 0));
  REFUSED(g(C, 64, (1ll << 30) + 1, 64, 64, 8, nullptr, nullptr, X, 8), OQ_ERR_UNSUPPORTED);
  REFUSED(g(C, 64, -1, 64, 64, 8, nullptr, nullptr, X, 8), OQ_ERR_INVALID_ARG);
  REFUSED(g(C, 64, 4, 72, 64, 8, nullptr, nullptr, X, 8), OQ_ERR_UNSUPPORTED);
  REFUSED(g(C, 64, 4, 131072, 64, 8, nullptr, nullptr, X, 8), OQ_ERR_UNSUPPORTED);
  REFUSED(g(C, 64, 4, 64, 64, 8, F, nullptr, X, 8), OQ_ERR_INVALID_ARG);
  REFUSED(g(C, 48, 4, 64, 64, 8, nullptr, nullptr, X, 8), OQ_ERR_INVALID_ARG);
  REFUSED(g(C, 64, 4, 64, (1 << 23) + 16, 8, nullptr, nullptr, X, 8), OQ_ERR_UNSUPPORTED);
  REFUSED(g(C4, 64, 4, 64, 64, 8, nullptr, nullptr, X, 8), OQ_ERR_ALIGNMENT);
  REFUSED(g(C, 64, 4, 64, 64, 8, F1, F, X, 8), OQ_ERR_ALIGNMENT);
  REFUSED(g(C, 64, 4, 64, 64, 8, nullptr, nullptr, X, 7), OQ_ERR_INVALID_ARG);
}

// T tokens of hq + hk heads of d, inputs and outputs with their own strides
int qk(int64_t T, int d, int hq, int hk, int64_t ld, int64_t hs, int64_t old, int64_t ohs, const oq_rope *r, const int32_t *pos,
       uint16_t *out = X, float eps = 1e-6f, const float *w = F) {
  return oq_qk_norm_rope(X, ld, hs, hq, X, ld, hs, hk, T, d, w, F, eps, r, pos, out, old, ohs, X, old, ohs, nullptr);
}

// no two heads of an output on one place, by counting
bool apart(int64_t ld, int64_t hs, int heads, int T, int d) {
  static unsigned char seen[1 << 16];
  std::memset(seen, 0, sizeof seen);
  for (int t = 0; t < T; ++t)
    for (int h = 0; h < heads; ++h)
      for (int e = 0; e < d; e += 8)
        if (seen[(t * ld + h * hs + e) / 8]++) return false;
  return true;
}

void heads() {
  const oq_rope rope{F, F, 100, 64, 0}, bad{F, nullptr, 100, 64, 0}, wide{F, F, 100, 136, 1};
  RUNS(qk(10, 128, 4, 2, 512, 128, 512, 128, &rope, nullptr), "heads");
  RUNS(qk(0x7fffffff, 512, 65535, 65535, 65535 * 512, 512, 65535 * 512, 512, &rope, I), "heads");
  RUNS(qk(0x7fffffff, 8, 65535, 1, INT64_MAX - 7, 8, INT64_MAX - 7, 8, nullptr, nullptr), "heads");
  RUNS(qk(10, 128, 4, 2, 128, 1280, 128, 1280, nullptr, nullptr), "heads");    // head after head
  RUNS(qk(10, 128, 4, 2, 128, 128, 512, 128, nullptr, nullptr), "heads");      // inputs may overlap
  RUNS(qk(1, 128, 4, 2, 0, 128, 0, 128, nullptr, nullptr), "heads");           // one token has no token stride
  RUNS(qk(10, 128, 1, 1, 128, 0, 128, 0, nullptr, nullptr), "heads");          // one head no head stride
  RUNS(qk(0, 128, 4, 2, 512, 128, 512, 128, &rope, nullptr), "heads");
  REFUSED(qk(101, 128, 4, 2, 512, 128, 512, 128, &rope, nullptr), OQ_ERR_INVALID_ARG);
  REFUSED(qk(1ll << 31, 128, 4, 2, 512, 128, 512, 128, nullptr, nullptr), OQ_ERR_UNSUPPORTED);
  REFUSED(qk(10, 128, 65536, 2, 512, 128, 512, 128, nullptr, nullptr), OQ_ERR_UNSUPPORTED);
  REFUSED(qk(10, 132, 4, 2, 1024, 136, 1024, 136, nullptr, nullptr), OQ_ERR_UNSUPPORTED);
  REFUSED(qk(10, 128, 4, 2, 512, 128, 512, 128, &bad, nullptr), OQ_ERR_INVALID_ARG);
  REFUSED(qk(10, 128, 4, 2, 512, 128, 512, 128, &wide, nullptr), OQ_ERR_INVALID_ARG);
  REFUSED(qk(10, 128, 4, 2, 512, 128, 512, 128, &rope, I1), OQ_ERR_ALIGNMENT);
  REFUSED(qk(10, 128, 4, 2, 512, 120, 512, 128, nullptr, nullptr), OQ_ERR_INVALID_ARG);
  REFUSED(qk(10, 128, 4, 2, 516, 128, 512, 128, nullptr, nullptr), OQ_ERR_ALIGNMENT);
  REFUSED(qk(10, 128, 4, 2, 512, 128, 512, 128, nullptr, nullptr, X4), OQ_ERR_ALIGNMENT);
  REFUSED(qk(10, 128, 4, 2, 512, 128, 512, 128, nullptr, nullptr, nullptr), OQ_ERR_INVALID_ARG);
  REFUSED(qk(10, 128, 4, 2, 512, 128, 512, 128, nullptr, nullptr, X, -1.f), OQ_ERR_INVALID_ARG);
  REFUSED(qk(10, 128, 4, 2, 512, 128, 512, 128, nullptr, nullptr, X, 1e-6f, F1), OQ_ERR_ALIGNMENT);
  // outputs: exactly the strides that keep every head apart
  for (int T : {2, 3, 5})
    for (int n : {2, 3, 4})
      for (int64_t ld = 16; ld <= 160; ld += 8)
        for (int64_t hs = 16; hs <= 160; hs += 8) {
          const int rc = qk(T, 16, n, 0, 1024, 16, ld, hs, nullptr, nullptr);
          TRUE((rc == OQ_OK) == apart(ld, hs, n, T, 16));
          TRUE(g_stub.launches == (rc == OQ_OK));
          g_stub.launches = 0;
          g_stub.last = "";
        }
}

oq_kv cache(int pages = 4, int page = 16, int heads = 8, int d = 128, int64_t stride = 0) {
  return oq_kv{X, X, stride ? stride : (int64_t)heads * page * d, pages, page, heads, d};
}

void append() {
  const oq_rope rope{F, F, 100, 64, 0};
  auto a = [&](int64_t T, const oq_kv &kv, int64_t ld, const oq_rope *r, const int64_t *slot, float eps = 0.f) {
    return oq_kv_append(X, ld, kv.d, X, ld, kv.d, T, F, eps, r, I, slot, &kv, nullptr);
  };
  RUNS(a(10, cache(), 1024, &rope, L), "heads_cache");
  RUNS(a(0x7fffffff, cache(0x7fffffff, 1024, 65535, 512), 65535 * 512, nullptr, L), "heads_cache");
  NOTHING(a(10, cache(0), 1024, &rope, L));
  REFUSED(oq_kv_append(X, 1024, 128, X, 1024, 128, 10, F, 0.f, nullptr, nullptr, L, nullptr, nullptr), OQ_ERR_INVALID_ARG);
  REFUSED(a(-1, cache(), 1024, &rope, L), OQ_ERR_INVALID_ARG);
  REFUSED(a(1ll << 31, cache(), 1024, &rope, L), OQ_ERR_UNSUPPORTED);
  REFUSED(a(10, cache(), 1024, &rope, nullptr), OQ_ERR_INVALID_ARG);
  REFUSED(a(10, cache(), 1024, &rope, L4), OQ_ERR_ALIGNMENT);
  REFUSED(a(10, cache(), 1020, &rope, L), OQ_ERR_ALIGNMENT);
  REFUSED(a(10, cache(), 1024, &rope, L, INFINITY), OQ_ERR_INVALID_ARG);
  REFUSED(a(10, cache(-1), 1024, &rope, L), OQ_ERR_INVALID_ARG);
  REFUSED(a(10, cache(4, 12), 1024, &rope, L), OQ_ERR_UNSUPPORTED);
  REFUSED(a(10, cache(4, 16, 65536, 8), 65536 * 8, nullptr, L), OQ_ERR_UNSUPPORTED);
  REFUSED(a(10, cache(4, 16, 8, 128, 8), 1024, &rope, L), OQ_ERR_INVALID_ARG);
  REFUSED(a(10, cache(4, 1024, 65535, 0x7fffffff, INT64_MAX - 7), 1024, &rope, L), OQ_ERR_UNSUPPORTED);  // a page of 2^57 elements
  REFUSED(a(10, cache(4, 16, 8, 520), 8 * 520, nullptr, L), OQ_ERR_UNSUPPORTED);
}

struct At {
  int B = 4, n_q = 1, heads_q = 32, prefix = 60, table_ld = 2;
  oq_kv kv = cache();
  const int32_t *pt = I, *tables = I, *lens = I;
  float scale = 0.1f;
  uint16_t *q = X, *o = X;
  int64_t ld = 4096, o_ld = 4096, o_hs = 128;
  float *lse = nullptr;
  void *ws = g_buf;
  size_t ws_bytes = ALL;
};
int call(const At &a) {
  return oq_attn_prefix(a.q, a.ld, a.kv.d, a.B, a.n_q, a.heads_q, &a.kv, a.pt, a.prefix, a.tables, a.table_ld, a.lens, a.scale, a.o,
                        a.o_ld, a.o_hs, a.lse, a.ws, a.ws_bytes, nullptr);
}
size_t ws_of(const At &a) { return oq_attn_prefix_ws_bytes(a.B, a.n_q, a.heads_q, &a.kv, a.prefix, a.table_ld); }

void attention() {
  const At d;
  auto with = [&](auto set) { At a = d; set(a); return a; };
#define REFUSED_WITH(change, code) REFUSED(call(with([](At &a) { change; })), code)
#define RUNS_WITH(change) RUNS(call(with([](At &a) { change; })), "attn_prefix")
  RUNS(call(d), "attn_prefix");
  RUNS_WITH(a.pt = nullptr; a.prefix = 0);
  RUNS_WITH(a.tables = nullptr; a.lens = nullptr; a.table_ld = 0);
  RUNS_WITH(a.scale = -2.3e38f);
  RUNS_WITH(a.scale = 0.f);
  RUNS_WITH(a.kv = cache(0); a.kv.k = nullptr; a.kv.v = nullptr; a.ws = nullptr);  // no page: every row is empty
  NOTHING(call(with([](At &a) { a.B = 0; a.q = nullptr; a.o = nullptr; a.ws = nullptr; })));
  // a workspace that is missing or a byte short
  const size_t need = ws_of(d);
  TRUE(need > 0);
  REFUSED_WITH(a.ws = nullptr, OQ_ERR_WORKSPACE);
  REFUSED(call(with([&](At &a) { a.ws_bytes = need - 1; })), OQ_ERR_WORKSPACE);
  REFUSED(call(with([&](At &a) { a.ws_bytes = 0; })), OQ_ERR_WORKSPACE);
  RUNS(call(with([&](At &a) { a.ws_bytes = need; })), "attn_prefix");
  // own keys alone, in one part: no workspace
  const At own = with([](At &a) { a.B = 64; a.prefix = 0; a.table_ld = 1; a.ws = nullptr; a.ws_bytes = 0; });
  TRUE(ws_of(own) == 0);
  RUNS(call(own), "attn_prefix");

  REFUSED(oq_attn_prefix(X, 4096, 128, 4, 1, 32, nullptr, I, 60, I, 2, I, 0.1f, X, 4096, 128, nullptr, g_buf, ALL, nullptr),
          OQ_ERR_INVALID_ARG);
  TRUE(oq_attn_prefix_ws_bytes(4, 1, 32, nullptr, 60, 2) == 0);
  REFUSED_WITH(a.B = -1, OQ_ERR_INVALID_ARG);
  REFUSED_WITH(a.n_q = 0, OQ_ERR_INVALID_ARG);
  REFUSED_WITH(a.heads_q = 30, OQ_ERR_INVALID_ARG);
  REFUSED_WITH(a.heads_q = 0, OQ_ERR_INVALID_ARG);
  REFUSED_WITH(a.kv = cache(4, 16, 8, 96), OQ_ERR_UNSUPPORTED);
  REFUSED_WITH(a.prefix = -1, OQ_ERR_INVALID_ARG);
  REFUSED_WITH(a.prefix = 0x7fffffff, OQ_ERR_UNSUPPORTED);
  REFUSED_WITH(a.table_ld = 1 << 27, OQ_ERR_UNSUPPORTED);
  REFUSED_WITH(a.table_ld = 0x7fffffff; a.kv = cache(4, 1024), OQ_ERR_UNSUPPORTED);
  REFUSED_WITH(a.B = 1 << 22; a.n_q = 1 << 21; a.heads_q = 1 << 21, OQ_ERR_UNSUPPORTED);
  REFUSED_WITH(a.B = 0x7fffffff; a.n_q = 0x7fffffff; a.heads_q = 0x7ffffff8, OQ_ERR_UNSUPPORTED);
  REFUSED_WITH(a.scale = 2.4e38f, OQ_ERR_INVALID_ARG);
  REFUSED_WITH(a.scale = NAN, OQ_ERR_INVALID_ARG);
  REFUSED_WITH(a.q = nullptr, OQ_ERR_INVALID_ARG);
  REFUSED_WITH(a.o = X4, OQ_ERR_ALIGNMENT);
  REFUSED_WITH(a.o_ld = 128; a.o_hs = 128, OQ_ERR_INVALID_ARG);
  REFUSED_WITH(a.pt = nullptr, OQ_ERR_INVALID_ARG);
  REFUSED_WITH(a.lens = nullptr, OQ_ERR_INVALID_ARG);
  REFUSED_WITH(a.tables = I1, OQ_ERR_ALIGNMENT);
  REFUSED_WITH(a.lse = F1, OQ_ERR_ALIGNMENT);
  REFUSED_WITH(a.ws = X4, OQ_ERR_ALIGNMENT);
}

// The plan of one call: chunks that cover the keys and fit the page numbers an
// item holds (with one to spare), items and workspace that follow from them.
void check_plan(const At &at) {
  if (at.B == 0) return;
  oq::AttnArgs a{};
  a.B = at.B;
  a.n_q = at.n_q;
  a.heads_q = at.heads_q;
  a.kv = at.kv;
  a.prefix_len = at.prefix;
  a.table_ld = at.table_ld;
  const oq::Plan p = oq::plan_for(a);
  const int G = a.heads_q / a.kv.heads;
  TRUE(p.rows == a.B * a.n_q * G && p.rows_all == (int64_t)p.rows * a.kv.heads);
  int parts = 0;
  for (int s = 0; s < 2; ++s) {
    const oq::PartPlan &q = p.launch.part[s];
    const int64_t keys = a.kv.pages == 0 ? 0 : s ? (int64_t)a.table_ld * a.kv.page : a.prefix_len;
    TRUE(q.part0 == parts && q.suffix == s && q.rows == p.rows);
    parts += q.splits;
    if (keys == 0) {
      TRUE(q.items == 0 && q.splits == 0);
      continue;
    }
    const int64_t rows = s ? a.n_q * G : p.rows, per = q.wide ? 256 : 32;
    TRUE((int64_t)q.tiles * per >= rows && ((int64_t)q.tiles - 1) * per < rows);
    TRUE(q.splits >= 1 && q.items == (int64_t)q.tiles * a.kv.heads * (s ? a.B : 1) * q.splits);
    const int64_t most = (int64_t)((q.wide ? oq::WIDE_PAGES : oq::NARROW_PAGES) - 1) * a.kv.page;
    const int tile = q.wide ? 64 : 32;
    TRUE(q.chunk > 0 && q.chunk % a.kv.page == 0 && q.chunk % tile == 0 && q.chunk <= most);
    if (!s) {
      TRUE((int64_t)q.splits * q.chunk >= keys && ((int64_t)q.splits - 1) * q.chunk < keys);
    } else {  // the kernel divides what a sequence has, n of the table's places
      for (int64_t n : {(int64_t)1, keys / 3 + 1, keys - 1 > 0 ? keys - 1 : 1, keys}) {
        const int64_t unit = a.kv.page > tile ? a.kv.page : tile;
        const int64_t even = ((n + q.splits - 1) / q.splits + unit - 1) / unit * unit, chunk = even > q.chunk ? even : q.chunk;
        TRUE(chunk <= most && chunk * q.splits >= n && chunk <= 0x7fffffff);
      }
    }
  }
  TRUE(p.parts == parts && p.launch.direct == (parts == 1));
  const size_t ws = ws_of(at);
  TRUE(ws == (parts == 1 ? 0 : (size_t)parts * (size_t)p.rows_all * ((size_t)a.kv.d * 4 + 8)));
}

void plans() {
  const int sizes[] = {0, 1, 31, 33, 64, 100, 255, 777, 2048, 5000, 32768, 131072, 1 << 20, 0x7fffffff - 1024};
  for (int cus : {1, 64, 256, 304}) {
    g_cus = cus;
    for (int page : {8, 64, 1024})
      for (int heads : {1, 8})
        for (int G : {1, 4, 40})
          for (int B : {1, 3, 64, 1000})
            for (int n_q : {1, 4, 100, 3000})
              for (int prefix : sizes)
                for (int own : sizes) {
                  At a;
                  a.B = B;
                  a.n_q = n_q;
                  a.heads_q = heads * G;
                  a.kv = cache(prefix % 5 ? 4 : 100, page, heads, G == 4 ? 64 : 128);
                  a.prefix = prefix;
                  a.table_ld = own / page;
                  check_plan(a);
                }
  }
  g_cus = 256;
  At a;  // the ends of the ranges
  for (int n_q : {1, 1 << 10, 1 << 27})
    for (int prefix : {0, 0x7fffffff - 1024})
      for (int places : {0, 0x7fffffff - 1024}) {
        a.n_q = n_q;
        a.heads_q = 8;
        a.B = (1 << 27) / n_q;
        a.prefix = prefix;
        a.table_ld = places / 16;
        check_plan(a);
      }
}

}  // namespace

int main() {
  weights();
  product();
  heads();
  append();
  attention();
  plans();
  if (g_fail) {
    std::printf("%d of %d cases failed\n", g_fail, g_cases);
    return 1;
  }
  std::printf("%d cases passed\n", g_cases);
  return 0;
}
