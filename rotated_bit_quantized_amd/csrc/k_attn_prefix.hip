// Attention of a batch that shares a prefix of a paged cache (oq_attn_prefix).
//
//   o = softmax(scale q K^T) V over the keys of the shared prefix and of the
//   row's own suffix, as one running softmax per part of the keys
//     m = max_j s_j,  l = sum_j 2^(s_j - m),  O = sum_j 2^(s_j - m) v_j
//   (s in units of log 2) and a join of the parts:
//     o = sum_p 2^(m_p - m) O_p / sum_p 2^(m_p - m) l_p,  m = max_p m_p.
//
// Rows of one key head are its query vectors in the order (token, query
// head): the prefix part takes them in tiles of 32 QT NW rows whatever
// sequence they belong to, so a prefix key is read once per tile; the suffix
// part takes the n_q G rows of one sequence.  A workgroup (NW wavefronts, 32
// QT rows each) walks a chunk of keys in tiles of KT through LDS, two
// buffers, copied global -> LDS while the other is used.  Both products run
// transposed on v_mfma_f32_32x32x16_bf16:
//   S^T[key][row] = K Q^T,   O^T[d][row] += V^T P^T,
// so that a lane owns one row: maximum, sum and rescaling are per-lane
// (one exchange between the lane's halves), and P^T leaves the first product
// in the layout that the second takes, up to an order of the keys that the
// V^T fragments (transposing LDS reads) follow.  The scale is applied to the
// float32 scores; P is rounded to bfloat16 for the second product, its sum l
// is not.  O is rescaled only when a row's maximum has grown by more than
// 2^8 since the last time (P then stays below 2^8, which costs float32 and
// bfloat16 no precision).
#include "oq_internal.h"

namespace oq {
namespace {

typedef short v8s __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int PAGES_MAX = 512;      // page numbers of one chunk, held in LDS
constexpr float RESCALE = 8.f;      // log2 growth of a maximum that rescales O
constexpr float LOG2E = 1.44269504088896340736f;
constexpr float LN2 = 0.69314718055994530942f;

// what masked key rows are copied from, so that they cannot put NaN into a product
__device__ const uint4 g_zero_row[16] = {};

// One launch's share of the work: the prefix (b < 0 side: table shared, rows
// of all sequences) or the suffixes (one sequence per item).
struct PartPlan {
  int suffix;     // 0 prefix, 1 suffixes
  int tiles;      // row tiles per key head (prefix) or per sequence and key head (suffix)
  int splits;     // chunks of the keys
  int chunk;      // keys per chunk: a multiple of KT and of the page (suffixes: the least)
  int part0;      // number of this launch's first part
  int rows;       // B n_q G, rows of one key head
  int64_t items;  // workgroups
  float c;        // log2(e) |scale|, or 1 where scale == 0
  uint32_t qand, qxor;  // on the bits of q pairs: sign of the scale, or zero
};

template <int D>
__device__ __forceinline__ int swz_k(int row) { return D == 128 ? row & 15 : (row >> 1) & 7; }
template <int D>
__device__ __forceinline__ int swz_v(int row) { return D == 128 ? (row & 3) << 2 : ((row >> 1) & 1) << 2; }

__device__ __forceinline__ float xhalf(float v) { return __shfl_xor(v, 32); }

template <int D, int NW, int QT, int KT>
__global__ void __launch_bounds__(64 * NW, NW == 4 && QT == 2 ? 1 : 2)
attn_part_kernel(const AttnArgs a, const PartPlan p, float *__restrict__ part_o, float2 *__restrict__ part_ml) {
  constexpr int KS = D / 16, DT = D / 32, SUB = KT / 32;
  constexpr int ROWB = 2 * D;              // bytes of a key row
  constexpr int TILE = KT * ROWB;          // bytes of a K or V tile
  constexpr int PIECES = TILE / 1024 / NW;  // 1 KiB copies per wavefront and tile
  static_assert(PIECES * NW * 1024 == TILE, "every wavefront copies the same share");
  __shared__ __attribute__((aligned(1024))) uint8_t s_kv[2][2 * TILE];
  __shared__ int s_page[PAGES_MAX];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r32 = lane & 31, half = lane >> 5;

  // Consecutive workgroups go to the 8 XCDs in turn; items that read the same
  // keys (the row tiles of one chunk) are consecutive, so give each XCD a run.
  int item = blockIdx.x;
  if (p.items % 8 == 0) item = (item & 7) * (int)(p.items >> 3) + (item >> 3);
  const int tile = item % p.tiles;
  item /= p.tiles;
  const int split = item % p.splits;
  item /= p.splits;
  const int hk = item % a.kv.heads, b = item / a.kv.heads;
  const int G = a.heads_q / a.kv.heads;

  // rows [r0, rend) of key head hk, keys [k0, n) of the part's places
  const int rbase = p.suffix ? b * a.n_q * G : 0;
  const int rend = p.suffix ? rbase + a.n_q * G : p.rows;
  const int r0 = rbase + tile * 32 * QT * NW + wave * 32 * QT;
  int chunk = p.chunk;
  int len = a.prefix_len, first = 0;  // row r sees places below min(n, len - first + token)
  const int32_t *table = a.prefix_table;
  int n = len;
  if (p.suffix) {
    table = a.tables + (int64_t)b * a.table_ld;
    const int cap = a.table_ld * a.kv.page;
    len = a.lens[b] > 0 ? a.lens[b] : 0;
    first = a.n_q - 1;
    // what the tile's last row sees
    int rl = rbase + (tile + 1) * 32 * QT * NW;
    if (rl > rend) rl = rend;
    const int64_t see = (int64_t)len - first + ((rl - 1) / G - b * a.n_q);
    n = see < 0 ? 0 : see < cap ? (int)see : cap;
    // the splits share what this sequence has, not what its table could hold
    const int unit = a.kv.page > KT ? a.kv.page : KT;
    const int even = ((n + p.splits - 1) / p.splits + unit - 1) / unit * unit;
    if (even > chunk) chunk = even;
  }
  const int64_t k0l = (int64_t)split * chunk;
  const int k0 = k0l < n ? (int)k0l : n;
  const int64_t prow = (int64_t)(p.part0 + split) * a.kv.heads * p.rows + (int64_t)hk * p.rows;
  if (k0 >= n) {
    if (half == 0)
#pragma unroll
      for (int t = 0; t < QT; ++t)
        if (r0 + 32 * t + r32 < rend) part_ml[prow + r0 + 32 * t + r32] = make_float2(-INFINITY, 0.f);
    return;
  }
  const int kend = n - k0 < chunk ? n : k0 + chunk;

  // the chunk's page numbers
  const int pl = __builtin_ctz((unsigned)a.kv.page);
  const int npages = ((kend - 1) >> pl) - (k0 >> pl) + 1;
  int bad = 0;
  for (int i = threadIdx.x; i < npages; i += 64 * NW) {
    const int pg = table[(k0 >> pl) + i];
    s_page[i] = pg;
    bad |= (unsigned)pg >= (unsigned)a.kv.pages;
  }
  const bool any_bad = __syncthreads_or(bad);

  const uint8_t *kb = reinterpret_cast<const uint8_t *>(a.kv.k + (int64_t)hk * a.kv.page * D);
  const uint8_t *vb = reinterpret_cast<const uint8_t *>(a.kv.v + (int64_t)hk * a.kv.page * D);
  const uint32_t lds0 = lds_addr_of(&s_kv[0][0]);
  auto issue = [&](int buf, int base) {
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      const int pos = (wave * PIECES + q) * 1024 + lane * 16;
      const int row = pos / ROWB, phys = (pos % ROWB) / 16;
      const int key = base + row;
      const int pg = key < kend ? s_page[(key - k0) >> pl] : -1;
      const int ck = 16 * (phys ^ swz_k<D>(row)), cv = 16 * (phys ^ swz_v<D>(row));
      const int64_t off = (int64_t)pg * (2 * a.kv.page_stride) + (key & (a.kv.page - 1)) * ROWB;
      const bool ok = (unsigned)pg < (unsigned)a.kv.pages;
      const uint8_t *zero = reinterpret_cast<const uint8_t *>(g_zero_row);
      const uint8_t *sk = ok ? kb + off + ck : zero + ck;
      const uint8_t *sv = ok ? vb + off + cv : zero + cv;
      const uint32_t dst = lds0 + buf * 2 * TILE + (wave * PIECES + q) * 1024;
      dma_lds16(sk, dst);
      dma_lds16(sv, dst + TILE);
    }
  };
  issue(0, k0);

  // this lane's rows: query fragments, number of places seen
  v8bf qf[QT][KS];
  int lim[QT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    int r = r0 + 32 * t + r32;
    if (r > rend - 1) r = rend - 1;
    const int tok = r / G, h = hk * G + (r - tok * G);
    const int64_t see = p.suffix ? (int64_t)len - first + (tok - b * a.n_q) : n;
    lim[t] = see < kend ? (int)see : kend;
    const uint16_t *src = a.q + tok * a.q_ld + h * a.q_hs + 8 * half;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      u32x4 v = *reinterpret_cast<const u32x4 *>(src + 16 * ks);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = (v[e] & p.qand) ^ p.qxor;
      qf[t][ks] = __builtin_bit_cast(v8bf, v);
    }
  }

  v16f O[QT][DT];
  float m[QT], l[QT];
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    m[t] = -INFINITY;
    l[t] = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d) O[t][d] = (v16f){};
  }
  const int steps = (kend - k0 + KT - 1) / KT;
  for (int st = 0; st < steps; ++st) {
    __builtin_amdgcn_s_waitcnt(0x0F70);  // this wavefront's copies of the tile have landed
    asm volatile("" ::: "memory");
    if (NW > 1) __builtin_amdgcn_s_barrier();  // and everybody's; nobody reads the other buffer any more
    asm volatile("" ::: "memory");
    const int base = k0 + st * KT;
    if (st + 1 < steps) issue((st + 1) & 1, base + KT);
    const uint8_t *tk = s_kv[st & 1], *tv = s_kv[st & 1] + TILE;

    v16f S[QT][SUB];
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
#pragma unroll
      for (int t = 0; t < QT; ++t) S[t][u] = (v16f){};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int row = 32 * u + r32;
        const v8bf kf = *reinterpret_cast<const v8bf *>(tk + row * ROWB + 16 * ((2 * ks + half) ^ swz_k<D>(row)));
#pragma unroll
        for (int t = 0; t < QT; ++t) S[t][u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[t][ks], S[t][u], 0, 0, 0);
      }
    }

    // the keys of the tile that are there: below kend, on a page of the cache
    const bool masked = any_bad || base + KT > kend;
    uint64_t there = ~0ull;
    if (masked) {
      const int key = base + lane;
      there = __ballot(key < kend && (unsigned)s_page[(key < kend ? key - k0 : 0) >> pl] < (unsigned)a.kv.pages);
    }

    v8bf pf[QT][2 * SUB];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      if (masked || !__all(base + KT <= lim[t])) {
        // bit 4 half + 8 (e >> 2) + (e & 3) of word u: element e's key is there and seen
        const int seen = lim[t] - base;
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
          const int s = seen - 32 * u;
          uint32_t bits = (uint32_t)(there >> (32 * u)) & (s >= 32 ? ~0u : s <= 0 ? 0u : (1u << s) - 1u);
          bits >>= 4 * half;
#pragma unroll
          for (int e = 0; e < 16; ++e) S[t][u][e] = (bits >> (8 * (e >> 2) + (e & 3))) & 1u ? S[t][u][e] : -INFINITY;
        }
      }
      float mx = S[t][0][0];
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int e = 0; e < 16; ++e) mx = __builtin_elementwise_maximum(mx, S[t][u][e]);
      mx = fmaxf(mx, xhalf(mx)) * p.c;
      if (__any(mx > m[t] + RESCALE)) {
        const float mn = fmaxf(m[t], mx);
        const float al = mn == -INFINITY ? 1.f : exp2f(m[t] - mn);
        m[t] = mn;
        l[t] *= al;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int e = 0; e < 16; ++e) O[t][d][e] *= al;
      }
      const float mu = m[t] == -INFINITY ? 0.f : m[t];
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(S[t][u][e], p.c, -mu));
          l[t] += x;
          pf[t][2 * u + (e >> 3)][e & 7] = (__bf16)x;
        }
    }

#pragma unroll
    for (int kk = 0; kk < 2 * SUB; ++kk) {
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        v8s vf;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int row = 16 * kk + 8 * w + 4 * half + ((lane & 15) >> 2);
          const int c = 4 * d + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
          const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) v4s *)(tv + row * ROWB + 16 * (c ^ swz_v<D>(row)) + 8 * (lane & 1)));
#pragma unroll
          for (int e = 0; e < 4; ++e) vf[4 * w + e] = x[e];
        }
#pragma unroll
        for (int t = 0; t < QT; ++t)
          O[t][d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, vf), pf[t][kk], O[t][d], 0, 0, 0);
      }
    }
    if (NW == 1) __builtin_amdgcn_s_waitcnt(0xC07F);  // reads of this buffer are done before its next copies
  }

#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const int r = r0 + 32 * t + r32;
    const float lt = l[t] + xhalf(l[t]);
    if (r >= rend) continue;
    if (half == 0) part_ml[prow + r] = make_float2(m[t], lt);
    float *dst = part_o + (prow + r) * D + 4 * half;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<float4 *>(dst + 32 * d + 8 * e) =
            make_float4(O[t][d][4 * e], O[t][d][4 * e + 1], O[t][d][4 * e + 2], O[t][d][4 * e + 3]);
  }
}

// The join: D / 4 lanes per row.
template <int D>
__global__ void __launch_bounds__(256)
attn_join_kernel(const AttnArgs a, int rows, int parts, const float *__restrict__ part_o, const float2 *__restrict__ part_ml) {
  constexpr int L = D / 4;
  const int64_t all = (int64_t)rows * a.kv.heads;
  const int64_t id = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  const int gl = threadIdx.x % L;
  if (id >= all) return;
  float m = -INFINITY;
  for (int s = 0; s < parts; ++s) {
    const float2 v = part_ml[s * all + id];
    m = fmaxf(m, v.x);
  }
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (m != -INFINITY) {
    for (int s = 0; s < parts; ++s) {
      const float2 v = part_ml[s * all + id];
      if (v.y == 0.f) continue;  // no keys: its O is not written
      const float w = exp2f(v.x - m);
      const float4 x = *reinterpret_cast<const float4 *>(part_o + (s * all + id) * D + 4 * gl);
      l = __builtin_fmaf(w, v.y, l);
      o.x = __builtin_fmaf(w, x.x, o.x);
      o.y = __builtin_fmaf(w, x.y, o.y);
      o.z = __builtin_fmaf(w, x.z, o.z);
      o.w = __builtin_fmaf(w, x.w, o.w);
    }
  }
  const int G = a.heads_q / a.kv.heads;
  const int hk = (int)(id / rows), r = (int)(id - (int64_t)hk * rows);
  const int tok = r / G, h = hk * G + (r - tok * G);
  const float inv = m == -INFINITY ? 0.f : 1.f / l;
  uint2 y;
  y.x = (uint32_t)f32_to_bf16_rne(o.x * inv) | ((uint32_t)f32_to_bf16_rne(o.y * inv) << 16);
  y.y = (uint32_t)f32_to_bf16_rne(o.z * inv) | ((uint32_t)f32_to_bf16_rne(o.w * inv) << 16);
  *reinterpret_cast<uint2 *>(a.o + tok * a.o_ld + h * a.o_hs + 4 * gl) = y;
  if (a.lse && gl == 0) a.lse[(int64_t)tok * a.heads_q + h] = m == -INFINITY ? -INFINITY : LN2 * (m + log2f(l));
}

// Row tile shape: wavefronts and 32-row blocks per wavefront.
struct Shape {
  int nw, qt, kt;
  int rows() const { return 32 * nw * qt; }
};

Shape shape_for(int rows) {
  if (rows <= 32) return {1, 1, 32};
  if (rows <= 64) return {2, 1, 64};
  if (rows <= 128) return {4, 1, 64};
  return {4, 2, 64};
}

struct Plan {
  PartPlan part[2];
  Shape shape[2];
  int parts;
  int64_t rows_all;
};

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

Plan plan_for(const AttnArgs &a) {
  Plan p;
  const int G = a.heads_q / a.kv.heads;
  const int rows = a.B * a.n_q * G;
  p.rows_all = (int64_t)rows * a.kv.heads;
  p.parts = 0;
  for (int s = 0; s < 2; ++s) {
    PartPlan &q = p.part[s];
    const int64_t keys = a.kv.pages == 0 ? 0 : s ? (int64_t)a.table_ld * a.kv.page : a.prefix_len;
    const int group_rows = s ? a.n_q * G : rows;
    const Shape sh = p.shape[s] = shape_for(group_rows);
    q.suffix = s;
    q.rows = rows;
    q.part0 = p.parts;
    q.tiles = (group_rows + sh.rows() - 1) / sh.rows();
    q.splits = 0;
    q.items = 0;
    q.chunk = 0;
    if (keys == 0) continue;
    const int64_t unit = a.kv.page > sh.kt ? a.kv.page : sh.kt;
    const int64_t groups = (int64_t)q.tiles * a.kv.heads * (s ? a.B : 1);
    // enough workgroups for every CU: 1 of 4 wavefronts with 64 rows each, 8 single ones
    const int64_t want = (int64_t)device_cus() * (sh.nw == 4 ? (sh.qt == 2 ? 1 : 2) : sh.nw == 2 ? 4 : 8);
    int64_t splits = want / groups;
    if (splits < 1) splits = 1;
    int64_t chunk = round_up((keys + splits - 1) / splits, unit);
    const int64_t most = (int64_t)(PAGES_MAX - 1) * a.kv.page / unit * unit;
    if (chunk > most) chunk = most;
    q.splits = (int)((keys + chunk - 1) / chunk);
    q.chunk = (int)(s ? unit : chunk);
    q.items = groups * q.splits;
    p.parts += q.splits;
  }
  return p;
}

template <int D, int NW, int QT, int KT>
hipError_t launch_part(const AttnArgs &a, const PartPlan &p, float *po, float2 *pm, hipStream_t stream) {
  hipLaunchKernelGGL((attn_part_kernel<D, NW, QT, KT>), dim3((unsigned)p.items), dim3(64 * NW), 0, stream, a, p, po, pm);
  return hipGetLastError();
}

template <int D>
hipError_t launch_d(const AttnArgs &a, const Plan &p, float *po, float2 *pm, hipStream_t stream) {
  for (int s = 0; s < 2; ++s) {
    if (!p.part[s].items) continue;
    if (p.part[s].items > 0x7fffffff) return hipErrorInvalidConfiguration;
    const Shape sh = p.shape[s];
    const hipError_t e = sh.nw == 1   ? launch_part<D, 1, 1, 32>(a, p.part[s], po, pm, stream)
                         : sh.nw == 2 ? launch_part<D, 2, 1, 64>(a, p.part[s], po, pm, stream)
                         : sh.qt == 1 ? launch_part<D, 4, 1, 64>(a, p.part[s], po, pm, stream)
                                      : launch_part<D, 4, 2, 64>(a, p.part[s], po, pm, stream);
    if (e != hipSuccess) return e;
  }
  const int64_t per = 256 / (D / 4);
  hipLaunchKernelGGL((attn_join_kernel<D>), dim3((unsigned)((p.rows_all + per - 1) / per)), dim3(256), 0, stream, a,
                     p.part[0].rows, p.parts, po, pm);
  return hipGetLastError();
}

}  // namespace

size_t attn_prefix_ws(const AttnArgs &a) {
  const Plan p = plan_for(a);
  return (size_t)p.parts * (size_t)p.rows_all * ((size_t)a.kv.d * 4 + 8);
}

hipError_t launch_attn_prefix(const AttnArgs &a, void *ws, hipStream_t stream) {
  Plan p = plan_for(a);
  for (PartPlan &q : p.part) {
    q.c = a.scale == 0.f ? 1.f : __builtin_fabsf(a.scale) * LOG2E;
    q.qand = a.scale == 0.f ? 0u : 0xffffffffu;
    q.qxor = a.scale < 0.f ? 0x80008000u : 0u;
  }
  float *po = static_cast<float *>(ws);
  float2 *pm = reinterpret_cast<float2 *>(po + (size_t)p.parts * p.rows_all * a.kv.d);
  return a.kv.d == 64 ? launch_d<64>(a, p, po, pm, stream) : launch_d<128>(a, p, po, pm, stream);
}

}  // namespace oq
