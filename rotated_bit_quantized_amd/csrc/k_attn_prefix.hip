// Attention of a batch that shares a prefix of a paged cache (oq_attn_prefix).
//
//   o = softmax(scale q K^T) V over the keys of the shared prefix and of the
//   row's own suffix, as one running softmax per part of the keys
//     m = max_j s_j,  l = sum_j 2^(s_j - m),  O = sum_j 2^(s_j - m) v_j
//   (s in units of log 2) and a join of the parts:
//     o = sum_p 2^(m_p - m) O_p / sum_p 2^(m_p - m) l_p,  m = max_p m_p.
//
// Rows of one key head are its query vectors in the order (token, query
// head): the prefix part takes them in tiles whatever sequence they belong to,
// so a prefix key is read once per tile; the suffix part takes the n_q G rows
// of one sequence.  An item is a row tile and a chunk of the keys, walked in
// tiles of keys.  Wide items: eight wavefronts of 32 rows share tiles of 64
// keys, K and V in rings of four LDS slots, copied global -> LDS two steps
// ahead, one barrier for two steps.  Narrow items: one wavefront of 32 rows,
// tiles of 32 keys, K fragments straight from memory, V through two LDS slots,
// no barrier at all.  Both kinds run in one launch, the join in a second (where
// there is more than one part).
// Both products run transposed on v_mfma_f32_32x32x16_bf16:
//   S^T[key][row] = K Q^T,   O^T[d][row] += V^T P^T,
// so that a lane owns one row: maximum, sum and rescaling are per-lane
// (one exchange between the lane's halves), and P^T leaves the first product
// in the layout that the second takes, up to an order of the keys that the
// V^T fragments (transposing LDS reads) follow.  The scale is applied to the
// float32 scores; P is rounded to bfloat16 for the second product, which takes
// both operands in V's type, its sum l is not.  That is the one place with fewer
// than 32 bits before the output's own rounding, and costs about as much as that:
// off by 0.0022 to 0.0024 of the norm against 64 bits, 0.0017 with P as two
// bfloat16 terms (and for exact results rounded once).  Two terms are half as
// many products again: 256 sequences over 32768 + 512 keys 214 -> 268 us, 8192
// tokens among themselves 568 -> 763.
// O is rescaled only when a row's maximum has grown by more than 2^8 since the
// last time (P then stays below 2^8, which costs float32 and bfloat16 no
// precision).
//
// What bounds it.  Wide items: the matrix and the vector unit together, a
// score costs 4 D operations on the one and an exponential, a fused multiply
// and add, an addition, half a maximum and half a conversion on the other, while
// every wavefront reads every K and V byte from LDS, at a clock that the power
// limits; 1024 rows of 8 heads over 32768 keys with D = 128 take 145 us, 0.95
// PFLOP/s (a large bf16 product of the library: 1.23).  Narrow items with long
// chunks: HBM, 16 sequences of 8000 keys each (524 MB) 103 us, 5.1 TB/s.  Short
// calls: latency, launch, page numbers, first keys, join; 3 sequences over
// 777 + 60 keys 9.8 us in all.
#include "attn_plan.h"

namespace oq {
namespace {

typedef short v8s __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float RESCALE = 8.f;      // log2 growth of a maximum that rescales O
constexpr float LN2 = 0.69314718055994530942f;

// what masked key rows are copied from, so that they cannot put NaN into a product
__device__ const uint4 g_zero_row[16] = {};

template <int D>
__device__ __forceinline__ int swz_k(int row) { return D == 128 ? row & 15 : (row >> 1) & 7; }
template <int D>
__device__ __forceinline__ int swz_v(int row) { return D == 128 ? (row & 3) << 2 : ((row >> 1) & 1) << 2; }

// the other half's value
__device__ __forceinline__ float xhalf(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(threadIdx.x & 32 ? r[0] : r[1]);
}

template <int C>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt(0x0F70 | (C & 0xF) | ((C >> 4) << 14));
}

// LDS of an item: K (wide items) and V slots, page numbers
template <int D, int NW>
struct Part {
  static constexpr int KT = NW == 1 ? 32 : 64;      // keys of a tile
  static constexpr int GRP = NW == 1 ? 1 : 2;       // steps between barriers
  static constexpr int RING = 2 * GRP;              // tile t of K and of V is in their slot t % RING
  static constexpr int TILE = KT * 2 * D;           // bytes of a K or V tile
  static constexpr int VBASE = NW == 1 ? 0 : RING;  // K slots, then V slots; one wavefront has K in registers
  static constexpr int PAGES_AT = (VBASE + RING) * TILE, PAGES_MAX = NW == 1 ? NARROW_PAGES : WIDE_PAGES;
  static constexpr int FLAG = PAGES_MAX - 1;        // place after the most page numbers of a chunk: see hide()
  static constexpr int LDS = PAGES_AT + 4 * PAGES_MAX;
};

template <int D, int NW>
__device__ __forceinline__ void part_body(const AttnArgs &a, const Launch &lp, const PartPlan &p, int item, uint8_t *smem,
                                          uint32_t spare, float *__restrict__ part_o, float2 *__restrict__ part_ml) {
  using P = Part<D, NW>;
  constexpr int KT = P::KT, GRP = P::GRP, RING = P::RING, TILE = P::TILE;
  constexpr int KS = D / 16, DT = D / 32, SUB = KT / 32;
  constexpr int ROWB = 2 * D;               // bytes of a key row
  constexpr int PIECES = TILE / 1024 / NW;  // 1 KiB copies per wavefront and K or V tile
  constexpr int PROWS = 1024 / ROWB;        // key rows of one: 4 or 8, on one page
  constexpr bool DK = NW == 1;              // K fragments straight from memory
  static_assert(PIECES * NW * 1024 == TILE, "every wavefront copies the same share");
  uint8_t *s_kv = smem;
  int *s_page = reinterpret_cast<int *>(smem + P::PAGES_AT);
  const int lane = threadIdx.x & 63, wave = NW == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r32 = lane & 31, half = lane >> 5;
  // the item's wavefronts meet; what they wrote to LDS is visible
  auto meet_lds = [&]() {
    if (NW > 1) {
      __syncthreads();
    } else {
      __builtin_amdgcn_s_waitcnt(0xC07F);
      __builtin_amdgcn_wave_barrier();
    }
    asm volatile("" ::: "memory");
  };

  // Consecutive workgroups go to the 8 XCDs in turn; items that read the same
  // keys (the row tiles of one chunk) are consecutive, so give each XCD a run.
  if (p.swizzle) item = (item & 7) * (int)(p.items >> 3) + (item >> 3);
  // A suffix's last rows see the most keys: they go first, so that what ends last
  // is short (8192 tokens among themselves 602 -> 537 us, 4096 180 -> 146, before hide() below).
  const int tile = p.suffix ? p.tiles - 1 - item % p.tiles : item % p.tiles;
  item /= p.tiles;
  const int split = item % p.splits;
  item /= p.splits;
  const int hk = item % a.kv.heads, b = item / a.kv.heads;
  const int G = a.heads_q / a.kv.heads;

  // rows [r0, rend) of key head hk, keys [k0, n) of the part's places
  const int rbase = p.suffix ? b * a.n_q * G : 0;
  const int rend = p.suffix ? rbase + a.n_q * G : p.rows;
  const int r0 = rbase + tile * 32 * NW + wave * 32;
  int chunk = p.chunk;
  int len = a.prefix_len, first = 0;  // row r sees places below min(n, len - first + token)
  const int32_t *table = a.prefix_table;
  int n = len, all_see = len;  // places below all_see are seen by every row of the item
  if (p.suffix) {
    table = a.tables + (int64_t)b * a.table_ld;
    const int cap = a.table_ld * a.kv.page;
    len = a.lens[b] > 0 ? a.lens[b] : 0;
    first = a.n_q - 1;
    // what the tile's last row sees
    int rl = rbase + (tile + 1) * 32 * NW;
    if (rl > rend) rl = rend;
    const int64_t see = (int64_t)len - first + ((rl - 1) / G - b * a.n_q);
    n = see < 0 ? 0 : see < cap ? (int)see : cap;
    const int64_t least = (int64_t)len - first + ((rbase + tile * 32 * NW) / G - b * a.n_q);
    all_see = least < 0 ? 0 : least < n ? (int)least : n;
    // the splits share what this sequence has, not what its table could hold
    const int unit = a.kv.page > KT ? a.kv.page : KT;
    const int64_t even = (((int64_t)n + p.splits - 1) / p.splits + unit - 1) / unit * unit;
    if (even > chunk) chunk = (int)even;
  }
  const int64_t k0l = (int64_t)split * chunk;
  const int k0 = k0l < n ? (int)k0l : n;
  const int64_t prow = (int64_t)(p.part0 + split) * a.kv.heads * p.rows + (int64_t)hk * p.rows;
  if (k0 >= n) {
    const int r = r0 + r32;
    if (r >= rend) return;
    if (!lp.direct) {
      if (half == 0) part_ml[prow + r] = make_float2(-INFINITY, 0.f);
      return;
    }
    const int tok = r / G, h = hk * G + (r - tok * G);
    uint16_t *dst = a.o + tok * a.o_ld + h * a.o_hs + half * (D / 2);
#pragma unroll
    for (int i = 0; i < D / 2; i += 8) *reinterpret_cast<u32x4 *>(dst + i) = (u32x4){};
    if (a.lse && half == 0) a.lse[(int64_t)tok * a.heads_q + h] = -INFINITY;
    return;
  }
  const int kend = n - k0 < chunk ? n : k0 + chunk;

  // the chunk's page numbers
  const int pl = __builtin_ctz((unsigned)a.kv.page);
  const int npages = ((kend - 1) >> pl) - (k0 >> pl) + 1;
  // every wavefront reads all of them and writes what the others write, so that
  // none has to wait for another
  int bad = 0;
  for (int i = lane; i < npages; i += 64) {
    const int pg = table[(k0 >> pl) + i];
    s_page[i] = pg;
    bad |= (unsigned)pg >= (unsigned)a.kv.pages;
  }
  const bool any_bad = __any(bad);
  __builtin_amdgcn_s_waitcnt(0xC07F);
  __builtin_amdgcn_wave_barrier();
  asm volatile("" ::: "memory");
  // Copies of tile t, this wavefront's pieces, K or V.  A piece is PROWS key
  // rows of one page, so its source is a scalar base and a fixed offset per
  // lane; the 16-byte chunks of a row are permuted by the row, on the source
  // side, against bank conflicts.
  const uint8_t *kb = reinterpret_cast<const uint8_t *>(a.kv.k + (int64_t)hk * a.kv.page * D);
  const uint8_t *vb = reinterpret_cast<const uint8_t *>(a.kv.v + (int64_t)hk * a.kv.page * D);
  const uint32_t lds0 = lds_addr_of(s_kv);
  const int prow_l = lane * 16 / ROWB, phys_l = lane * 16 % ROWB / 16;  // this lane's row and chunk of a piece
  const int steps = (kend - k0 + KT - 1) / KT;         // tiles
  const int full_steps = any_bad ? 0 : (kend - k0) / KT;  // those that have all their keys
  auto pages_of = [&](int t, int (&pg)[PIECES]) {
#pragma unroll
    for (int q = 0; q < PIECES; ++q) pg[q] = s_page[(t * KT + (wave * PIECES + q) * PROWS) >> pl];
  };
  // Without a branch, so that it can stand between products: where `full` is
  // false, page 0's first rows go to an unused KiB.
  auto copy_full = [&](bool full, bool is_v, int t, int q, int pg) {
    const int row = (wave * PIECES + q) * PROWS;
    const uint32_t c = 16 * (phys_l ^ (is_v ? swz_v<D>(row + prow_l) : swz_k<D>(row + prow_l)));
    const int64_t off = (int64_t)__builtin_amdgcn_readfirstlane(pg) * (2 * a.kv.page_stride) +
                        ((k0 + t * KT + row) & (a.kv.page - 1)) * ROWB;
    const uint32_t dst = ((is_v ? P::VBASE : 0) + t % RING) * TILE + (wave * PIECES + q) * 1024;
    dma_lds16_s((is_v ? vb : kb) + (full ? off : 0), prow_l * ROWB + c, full ? lds0 + dst : spare);
  };
  // A tile with missing keys: rows past the end and rows on a page outside the
  // cache are zeros, so that what no row sees, NaN perhaps, does not meet a zero
  // weight in the value product (nor does a seen infinity a second time).
  auto copy_any = [&](bool is_v, int t) {
    int pg[PIECES], key[PIECES];
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      key[q] = k0 + t * KT + (wave * PIECES + q) * PROWS + prow_l;
      const int at = key[q] < kend ? key[q] : kend - 1;
      pg[q] = s_page[(at - k0) >> pl];
    }
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      const int row = (wave * PIECES + q) * PROWS + prow_l;
      const uint32_t c = 16 * (phys_l ^ (is_v ? swz_v<D>(row) : swz_k<D>(row)));
      const uint8_t *at = (is_v ? vb : kb) + (int64_t)pg[q] * (2 * a.kv.page_stride) + (key[q] & (a.kv.page - 1)) * ROWB;
      const bool there = key[q] < kend && (unsigned)pg[q] < (unsigned)a.kv.pages;
      dma_lds16((there ? at : reinterpret_cast<const uint8_t *>(g_zero_row)) + c,
                lds0 + ((is_v ? P::VBASE : 0) + t % RING) * TILE + (wave * PIECES + q) * 1024);
    }
  };
#pragma unroll
  for (int t = 0; t <= GRP; ++t) {
    if (t < full_steps) {
      int pg[PIECES];
      pages_of(t, pg);
#pragma unroll
      for (int q = 0; q < PIECES; ++q) {
        if (!DK) copy_full(true, false, t, q, pg[q]);
        if (t < GRP) copy_full(true, true, t, q, pg[q]);
      }
    } else if (t < steps) {
      if (!DK) copy_any(false, t);
      if (t < GRP) copy_any(true, t);
    }
  }
  // Places that some rows of the item see and others do not (the query tokens'
  // own): a value there that is not finite would reach the others as 0 x NaN.
  // Each wavefront, before the tiles that it waited for are used, looks through
  // its pieces of them, makes such values zero and notes that there were some;
  // after the walk the rows that see them add them (reveal).  8 x 512 tokens among
  // themselves 47.7 -> 49.3 us, 8192 534 -> 538; single tokens have no such places.
  bool hidden = false;
  const bool ragged = all_see < kend;
  if (ragged && NW > 1) s_page[P::FLAG] = 0;
  auto hide = [&](int t) {
    if (!ragged || k0 + (t + 1) * KT <= all_see || t >= steps) return;
    u32x4 *at = reinterpret_cast<u32x4 *>(s_kv + (P::VBASE + t % RING) * TILE + wave * PIECES * 1024 + lane * 16);
    u32x4 v[PIECES];
#pragma unroll
    for (int q = 0; q < PIECES; ++q) v[q] = at[64 * q];
    uint32_t any = 0;  // an exponent of all ones carries into the sign's place
#pragma unroll
    for (int q = 0; q < PIECES; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) any |= (v[q][e] & 0x7f807f80u) + 0x00800080u;
    if (!(any & 0x80008000u)) return;
#pragma unroll
    for (int q = 0; q < PIECES; ++q) {
      if (k0 + t * KT + (wave * PIECES + q) * PROWS + prow_l < all_see) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t bad = ((v[q][e] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
        v[q][e] &= ~((bad >> 15) * 0xffffu);
        hidden |= bad != 0;
      }
      at[64 * q] = v[q];
    }
    if (NW > 1 && hidden) s_page[P::FLAG] = 1;
  };
  // K fragments of a tile in registers (DK): this lane's key row, chunks 2 ks +
  // half; past the end the last key, on a page outside the cache zeros
  v8bf kreg[DK ? KS : 1];
  typedef const __attribute__((address_space(1))) uint8_t *Global;  // else they become flat loads, which LDS reads wait for
  typedef const __attribute__((address_space(1))) v8bf *GlobalFrag;
  auto k_row = [&](int t) -> Global {
    int key = k0 + t * KT + r32;
    if (key > kend - 1) key = kend - 1;
    const int pg = s_page[(key - k0) >> pl];
    const uint8_t *at = kb + (int64_t)pg * (2 * a.kv.page_stride) + (key & (a.kv.page - 1)) * ROWB;
    return (Global)((unsigned)pg < (unsigned)a.kv.pages ? at : reinterpret_cast<const uint8_t *>(g_zero_row)) + 16 * half;
  };
  if (DK) {
    const Global at = k_row(0);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) kreg[ks] = *(GlobalFrag)(at + 32 * ks);
  }

  // this lane's row: query fragments, number of places seen
  v8bf qf[KS];
  int lim;
  {
    int r = r0 + r32;
    if (r > rend - 1) r = rend - 1;
    const int tok = r / G, h = hk * G + (r - tok * G);
    const int64_t see = p.suffix ? (int64_t)len - first + (tok - b * a.n_q) : n;
    lim = see < kend ? (int)see : kend;
    const uint16_t *src = a.q + tok * a.q_ld + h * a.q_hs + 8 * half;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      u32x4 v = *reinterpret_cast<const u32x4 *>(src + 16 * ks);
      if (lp.zero) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // an exponent of all ones carries into the sign's place
          const uint32_t bad = ((v[e] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
          v[e] = (bad >> 15) * 0x7fc0u;
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] ^= lp.qxor;
      qf[ks] = __builtin_bit_cast(v8bf, v);
    }
  }

  // fragment addresses: K row r32 of a 32-key block, chunk 2 ks + half; V keys
  // 16 kk + 8 w + 4 half + .. and d 32 dt + ..: a lane part that does not
  // change and a constant
  const uint8_t *k_at[DK ? 1 : KS], *v_at[DT];
  if (!DK) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) k_at[ks] = s_kv + r32 * ROWB + 16 * ((2 * ks + half) ^ swz_k<D>(r32));
  }
#pragma unroll
  for (int d = 0; d < DT; ++d) {
    const int row = 4 * half + ((lane & 15) >> 2), c = 4 * d + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    v_at[d] = s_kv + P::VBASE * TILE + row * ROWB + 16 * (c ^ swz_v<D>(row)) + 8 * (lane & 1);
  }
  auto k_frag = [&](int slot, int u, int ks) -> v8bf {
    return *reinterpret_cast<const v8bf *>(k_at[ks] + slot * TILE + 32 * u * ROWB);
  };
  auto v_frag = [&](int slot, int kk, int d) -> v8bf {
    v8s vf;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) v4s *)(v_at[d] + slot * TILE + (16 * kk + 8 * w) * ROWB));
#pragma unroll
      for (int e = 0; e < 4; ++e) vf[4 * w + e] = x[e];
    }
    return __builtin_bit_cast(v8bf, vf);
  };

  v16f O[DT];
  float m = -INFINITY, l[2] = {0.f, 0.f};
#pragma unroll
  for (int d = 0; d < DT; ++d) O[d] = (v16f){};

  // largest score of a lane in four chains
  float mq[4];
  auto max_of = [&](const v16f (&S)[SUB], int u, int e) {
    mq[e & 3] = u == 0 && e < 4 ? S[0][e] : __builtin_elementwise_maximum(mq[e & 3], S[u][e]);
  };
  auto max_all = [&](const v16f (&S)[SUB]) {
#pragma unroll
    for (int u = 0; u < SUB; ++u)
#pragma unroll
      for (int e = 0; e < 16; ++e) max_of(S, u, e);
  };
  // Masks the scores of tile `base` where it needs it and moves the reference m
  // (with O and l) where a row's maximum has outgrown it.
  auto settle = [&](v16f (&S)[SUB], int base) {
    if (any_bad || !__all(base + KT <= lim)) {
      // the keys of the tile that are there: below kend, on a page of the cache
      const int key = base + lane;
      const uint64_t there =
          __ballot(key < kend && (unsigned)s_page[(key < kend ? key - k0 : 0) >> pl] < (unsigned)a.kv.pages);
      // bit 8 (e >> 2) + (e & 3) of a word: element e's key is there and seen
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        const int s = lim - base - 32 * u;
        uint32_t bits = (uint32_t)(there >> (32 * u)) & (s >= 32 ? ~0u : s <= 0 ? 0u : (1u << s) - 1u);
        bits >>= 4 * half;
#pragma unroll
        for (int e = 0; e < 16; ++e) S[u][e] = (bits >> (8 * (e >> 2) + (e & 3))) & 1u ? S[u][e] : -INFINITY;
      }
      max_all(S);
    }
    float mx = __builtin_elementwise_maximum(__builtin_elementwise_maximum(mq[0], mq[1]),
                                             __builtin_elementwise_maximum(mq[2], mq[3]));
    mx = fmaxf(mx, xhalf(mx)) * lp.c;
    if (__any(mx > m + RESCALE)) {
      const float mn = mx > m + RESCALE ? mx : m;  // a row's own decision: its result does not depend on the others
      const float al = mn == -INFINITY ? 1.f : exp2f(m - mn);
      m = mn;
      l[0] *= al;
      l[1] *= al;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) O[d][e] *= al;
    }
  };

  // scores of the first tile
  wait_vm<0>();
  asm volatile("" ::: "memory");
  meet_lds();
  v16f S[SUB], T[SUB];  // scores of two tiles in turn
#pragma unroll
  for (int u = 0; u < SUB; ++u) {
    S[u] = (v16f){};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      S[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(DK ? kreg[ks] : k_frag(0, u, ks), qf[ks], S[u], 0, 0, 0);
  }
  if (DK) {
    const Global at = k_row(1);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) kreg[ks] = *(GlobalFrag)(at + 32 * ks);
  }
  max_all(S);
  settle(S, k0);

  // Step t: scores of tile t + 1 and the value product of tile t, its softmax
  // numerators formed in between, so that the matrix and the vector units work
  // at the same time.  Per 32 keys KS + 2 DT products, each with its fragment
  // read AHEAD products before and, after it, its share of the numerators
  // (pairs of them; those of 8 keys per half wave, 4 pairs, are due before the
  // first product that takes them) and of the next copies.
  constexpr int PER = KS + 2 * DT, SLOTS = SUB * PER, PAIRS = 8 * SUB, AHEAD = 3;
  auto step = [&](auto slot, int t0, const v16f (&S)[SUB], v16f (&Sn)[SUB]) {
    constexpr int v_slot = slot, ks_slot = (v_slot + 1) % RING;  // t0 % RING
    const int tk = t0 + GRP + 1, tv = t0 + GRP;  // the tiles to copy, where they have all their keys
    const bool full_k = tk < full_steps, full_v = tv < full_steps;
    int pgk[PIECES], pgv[PIECES];
    if (!DK) pages_of(full_k ? tk : 0, pgk);
    pages_of(full_v ? tv : 0, pgv);
    const Global k_next = DK ? k_row(t0 + 2) : nullptr;
    const float mu = m == -INFINITY ? 0.f : m;
    v8bf pf[2 * SUB], frag[AHEAD + 1];
    auto frag_of = [&](int t) -> v8bf {
      const int u = t / PER, w = t % PER;
      return w < KS ? (DK ? kreg[w] : k_frag(ks_slot, u, w)) : v_frag(v_slot, 2 * u + (w - KS) / DT, (w - KS) % DT);
    };
    // a wavefront by itself sends them at once, so that they have the whole step
    if (DK && full_v) {
#pragma unroll
      for (int q = 0; q < PIECES; ++q) copy_full(true, true, tv, q, pgv[q]);
    }
#pragma unroll
    for (int t = 0; t < AHEAD; ++t) frag[t] = frag_of(t);
#pragma unroll
    for (int t = 0; t < SLOTS; ++t) {
      if (t + AHEAD < SLOTS) frag[(t + AHEAD) % (AHEAD + 1)] = frag_of(t + AHEAD);
      const int u = t / PER, w = t % PER;
      const v8bf f = frag[t % (AHEAD + 1)];
      if (w < KS) {
        Sn[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, qf[w], w == 0 ? (v16f){} : Sn[u], 0, 0, 0);
        if (DK) kreg[w] = *(GlobalFrag)(k_next + 32 * w);
      } else {
        const int kk = 2 * u + (w - KS) / DT, d = (w - KS) % DT;
        O[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, pf[kk], O[d], 0, 0, 0);
      }
      // a 32 keys' scores stand two products after their last: their maximum
#pragma unroll
      for (int e = 0; e < 16; ++e)
#pragma unroll
        for (int x = 0; x < SUB; ++x)
          if (t == x * PER + KS + 2 + e * (2 * DT - 2) / 16) max_of(Sn, x, e);
      constexpr int RATE = D == 64 ? 4 : 2;  // thirds of a pair per product
#pragma unroll
      for (int pr = t * RATE / 3 + (t > 0); pr < (t + 1) * RATE / 3 + 1 && pr < PAIRS; ++pr) {
        const int pu = pr / 8, e = 2 * (pr % 8);
        const float x0 = __builtin_amdgcn_exp2f(__builtin_fmaf(S[pu][e], lp.c, -mu));
        const float x1 = __builtin_amdgcn_exp2f(__builtin_fmaf(S[pu][e + 1], lp.c, -mu));
        l[0] += x0;
        l[1] += x1;
        pf[2 * pu + (e >> 3)][e & 7] = (__bf16)x0;
        pf[2 * pu + (e >> 3)][(e & 7) + 1] = (__bf16)x1;
      }
#pragma unroll
      for (int q = 0; q < PIECES; ++q) {
        if (!DK && t == 2 + 2 * q * (SLOTS - 4) / (2 * PIECES)) copy_full(full_k, false, tk, q, pgk[q]);
        if (!DK && t == 2 + (2 * q + 1) * (SLOTS - 4) / (2 * PIECES)) copy_full(full_v, true, tv, q, pgv[q]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // GRP (1 or 2) steps between barriers: the tiles that they read have landed
  // before, the copies that they send go to slots that nobody reads any more.
  auto meet = [&](int t0) {
    wait_vm<0>();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int t = 0; t < GRP; ++t) hide(t0 + t);
    meet_lds();
    __builtin_amdgcn_sched_barrier(0);
    // the copies that the steps do not send: tiles with missing keys
    if (t0 + 2 * GRP >= full_steps) {
      for (int t = t0 + GRP; t <= t0 + 2 * GRP; ++t) {
        if (t < full_steps || t >= steps) continue;
        if (!DK && t > t0 + GRP) copy_any(false, t);
        if (t < t0 + 2 * GRP) copy_any(true, t);
      }
    }
  };
  using Int0 = std::integral_constant<int, 0>;
  using Int1 = std::integral_constant<int, 1>;
  using Int2 = std::integral_constant<int, 2 % RING>;
  using Int3 = std::integral_constant<int, 3 % RING>;
  for (int t0 = 0; t0 < steps;) {
    meet(t0);
    step(Int0{}, t0, S, T);
    if (++t0 == steps) break;
    settle(T, k0 + t0 * KT);
    if (GRP == 1) meet(t0);
    step(Int1{}, t0, T, S);
    if (++t0 == steps) break;
    settle(S, k0 + t0 * KT);
    if (RING == 2) continue;
    meet(t0);
    step(Int2{}, t0, S, T);
    if (++t0 == steps) break;
    settle(T, k0 + t0 * KT);
    step(Int3{}, t0, T, S);
    if (++t0 == steps) break;
    settle(S, k0 + t0 * KT);
  }
  if (!DK) wait_vm<0>();  // no copy outlives the item; one wavefront's have all been used

  // reveal: what hide() has taken out, for the rows that see it (whatever its
  // weight, an infinity stays one and NaN is NaN)
  if (ragged && (NW > 1 ? s_page[P::FLAG] != 0 : __any(hidden))) {
    for (int key = all_see > k0 ? all_see : k0; key < lim; ++key) {
      const int pg = s_page[(key - k0) >> pl];
      if ((unsigned)pg >= (unsigned)a.kv.pages) continue;
      const uint8_t *at = vb + (int64_t)pg * (2 * a.kv.page_stride) + (key & (a.kv.page - 1)) * ROWB + 8 * half;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint2 v = *reinterpret_cast<const uint2 *>(at + 64 * d + 16 * e);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float f = x & 1 ? bf16_hi(x < 2 ? v.x : v.y) : bf16_lo(x < 2 ? v.x : v.y);
            O[d][4 * e + x] += __builtin_isfinite(f) ? 0.f : f;
          }
        }
    }
  }

  const int r = r0 + r32;
  const float ls = l[0] + l[1], lt = ls + xhalf(ls);
  if (r >= rend) return;
  if (lp.direct) {  // what the join of one part would give
    const int tok = r / G, h = hk * G + (r - tok * G);
    const bool none = lt == 0.f;  // no key has weight: zeros, whatever the values were
    const float inv = 1.f / lt;
    auto out = [&](float v) { return (uint32_t)f32_to_bf16_rne(none ? 0.f : v * inv); };
    uint16_t *dst = a.o + tok * a.o_ld + h * a.o_hs + 4 * half;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<uint2 *>(dst + 32 * d + 8 * e) =
            make_uint2(out(O[d][4 * e]) | out(O[d][4 * e + 1]) << 16, out(O[d][4 * e + 2]) | out(O[d][4 * e + 3]) << 16);
    if (a.lse && half == 0) a.lse[(int64_t)tok * a.heads_q + h] = none ? -INFINITY : LN2 * (m + log2f(lt));
    return;
  }
  // a sum that is NaN reaches the output whatever m, which NaN scores do not move
  if (half == 0) part_ml[prow + r] = make_float2(lt == lt ? m : 0.f, lt);
  float *dst = part_o + (prow + r) * D + 4 * half;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<float4 *>(dst + 32 * d + 8 * e) =
          make_float4(O[d][4 * e], O[d][4 * e + 1], O[d][4 * e + 2], O[d][4 * e + 3]);
}

template <int D>
__global__ void __launch_bounds__(512, 2)
attn_part_kernel(const AttnArgs a, const Launch lp, float *__restrict__ part_o, float2 *__restrict__ part_ml) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const uint32_t spare = lds_addr_of(smem);  // a KiB that nobody reads
  uint8_t *mine = smem + 1024;
  const int past = (int)blockIdx.x - lp.lead;
  if (past >= 0 && past < lp.wide_items) {
    const int first = lp.part[0].wide ? (int)lp.part[0].items : 0;
    const int w = past >= first;
    part_body<D, 8>(a, lp, lp.part[w], w ? past - first : past, mine, spare, part_o, part_ml);
  } else {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int item = (past < 0 ? (int)blockIdx.x : (int)blockIdx.x - lp.wide_items) * lp.waves + wave;
    if (item >= lp.narrow_items) return;
    const int first = lp.part[0].wide ? 0 : (int)lp.part[0].items;
    const int w = item >= first;
    part_body<D, 1>(a, lp, lp.part[w], w ? item - first : item, mine + wave * Part<D, 1>::LDS, spare, part_o, part_ml);
  }
}

// a value's partners at lane distances 1, 2, the rest of 8, of 16, 32 and 64
template <class F>
__device__ __forceinline__ float wave_all(float v, F f) {
  auto dpp = [&](auto ctrl) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  v = f(v, dpp(std::integral_constant<int, 0xB1>{}));
  v = f(v, dpp(std::integral_constant<int, 0x4E>{}));
  v = f(v, dpp(std::integral_constant<int, 0x141>{}));
  v = f(v, dpp(std::integral_constant<int, 0x140>{}));
  v = f(v, __shfl_xor(v, 16));
  return f(v, xhalf(v));
}

// The join: lanes hold the parts' statistics, 64 parts at a time; D / 4 lanes
// then take a part's O each, 256 / D parts at once.  Latency bounds it where
// there are few rows: there the first BATCH loads of O leave beside those of the
// statistics, whatever their weights (what a part without keys has left unwritten
// is dropped), and with WAVES = 4 four wavefronts share a row, all of 64 parts'
// loads on their way at once, and their sums meet in LDS.  1 sequence, 32 rows, 64
// parts: 20 us with the parts' kernel, 28 with a wavefront a row.  96 rows, 14
// parts: 3.8 us against 5.6 without the early loads.  Where there are many rows
// the traffic counts, and parts without keys are not read (WAVES = 0): 8192 rows
// 9.7 us, 11.4 with early loads.
template <int D, int WAVES>
__global__ void __launch_bounds__(256)
attn_join_kernel(const AttnArgs a, int rows, int parts, const float *__restrict__ part_o, const float2 *__restrict__ part_ml) {
  constexpr int L = D / 4, AT = 64 / L, STEP = WAVES == 4 ? 4 * AT : AT;
  constexpr int BATCH = WAVES == 0 ? 0 : 64 / STEP < 8 ? 64 / STEP : 8;
  __shared__ float4 sum[WAVES == 4 ? 4 : 1][L];
  const int64_t all = (int64_t)rows * a.kv.heads;
  const int wave = threadIdx.x >> 6;
  const int64_t id = WAVES == 4 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + wave;
  const int lane = threadIdx.x & 63, gl = lane % L, sub = (WAVES == 4 ? wave * AT : 0) + lane / L;
  if (id >= all) return;
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float w, const float4 &v) {
    o.x = __builtin_fmaf(w, v.x, o.x);
    o.y = __builtin_fmaf(w, v.y, o.y);
    o.z = __builtin_fmaf(w, v.z, o.z);
    o.w = __builtin_fmaf(w, v.w, o.w);
  };
  auto stats = [&](int s) { return s < parts ? part_ml[s * all + id] : make_float2(-INFINITY, 0.f); };
  float2 next = stats(lane);
  for (int s0 = 0; s0 < parts; s0 += 64) {
    const int np = parts - s0 < 64 ? parts - s0 : 64;
    auto read = [&](int s) { return *reinterpret_cast<const float4 *>(part_o + ((s0 + s) * all + id) * D + 4 * gl); };
    float4 x[BATCH + 1];
    auto load = [&]() {
#pragma unroll
      for (int u = 0; u < BATCH; ++u)
        if (u * STEP < np) x[u] = read(u * STEP + sub < np ? u * STEP + sub : np - 1);
    };
    const float2 v = next;
    if (s0 == 0) load();
    next = stats(s0 + 64 + lane);
    const float mx = wave_all(v.x, [](float p, float q) { return fmaxf(p, q); });
    if (mx == -INFINITY) continue;  // no part of these has keys
    if (s0 > 0) load();
    const float mn = fmaxf(m, mx), al = exp2f(m - mn);
    m = mn;
    // -1: without keys, its O unwritten.  A weight that vanishes still takes its
    // part's O, which may be NaN.
    const float w = v.y == 0.f ? -1.f : exp2f(v.x - m);
    l = l * al + wave_all(w < 0.f ? 0.f : w * v.y, [](float p, float q) { return p + q; });
    o.x *= al, o.y *= al, o.z *= al, o.w *= al;
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      const float ws = __shfl(w, u * STEP + sub);  // lanes past the end have no keys either
      add(ws, ws < 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : x[u]);
    }
    for (int s = BATCH * STEP; s < np; s += STEP) {
      const float ws = __shfl(w, s + sub);
      if (ws >= 0.f) add(ws, read(s + sub));
    }
  }
#pragma unroll
  for (int x = L; x < 64; x <<= 1) {
    o.x += __shfl_xor(o.x, x);
    o.y += __shfl_xor(o.y, x);
    o.z += __shfl_xor(o.z, x);
    o.w += __shfl_xor(o.w, x);
  }
  if (WAVES == 4) {
    if (lane < L) sum[wave][lane] = o;
    __syncthreads();
    if (wave) return;
    o = sum[0][gl];
#pragma unroll
    for (int u = 1; u < 4; ++u) add(1.f, sum[u][gl]);
  }
  if (lane >= L) return;
  const int G = a.heads_q / a.kv.heads;
  const int hk = (int)(id / rows), r = (int)(id - (int64_t)hk * rows);
  const int tok = r / G, h = hk * G + (r - tok * G);
  const float inv = m == -INFINITY ? 0.f : 1.f / l;
  uint2 y;
  y.x = (uint32_t)f32_to_bf16_rne(o.x * inv) | ((uint32_t)f32_to_bf16_rne(o.y * inv) << 16);
  y.y = (uint32_t)f32_to_bf16_rne(o.z * inv) | ((uint32_t)f32_to_bf16_rne(o.w * inv) << 16);
  *reinterpret_cast<uint2 *>(a.o + tok * a.o_ld + h * a.o_hs + 4 * gl) = y;
  if (a.lse && lane == 0) a.lse[(int64_t)tok * a.heads_q + h] = m == -INFINITY ? -INFINITY : LN2 * (m + log2f(l));
}

template <int D>
hipError_t launch_d(const AttnArgs &a, Plan &p, float *po, float2 *pm, hipStream_t stream) {
  Launch &lp = p.launch;
  int64_t wide = 0, narrow = 0;
  for (PartPlan &q : lp.part) (q.wide ? wide : narrow) += q.items;
  if (wide + narrow > 0x7fffffff || (p.rows_all + 3) / 4 > 0x7fffffff) return hipErrorInvalidConfiguration;
  lp.wide_items = (int)wide;
  lp.narrow_items = (int)narrow;
  lp.waves = wide ? 8 : 1;
  // In two rounds, half of the single wavefronts' workgroups go first and half
  // last, so that their traffic and the wide items' products overlap: 256
  // sequences over 32768 + 512 keys 238 us (258 with all of them last).
  lp.lead = wide && !p.mixed ? (int)((narrow + 7) / 8 / 2) & ~7 : 0;
  for (PartPlan &q : lp.part) q.swizzle = q.items % 8 == 0 && (q.wide || lp.waves == 1);
  if (wide + narrow > 0) {
    constexpr int WIDE = Part<D, 8>::LDS, ONE = Part<D, 1>::LDS, MOST = (WIDE > 8 * ONE ? WIDE : 8 * ONE) + 1024;
    static_assert(MOST <= 160 * 1024, "LDS");
    static std::atomic<bool> attr_set[64];
    const hipError_t e = lds_limit_once((const void *)attn_part_kernel<D>, MOST, attr_set);
    if (e != hipSuccess) return e;
    const int lds = wide ? MOST : ONE + 1024;
    const int64_t blocks = wide + (narrow + lp.waves - 1) / lp.waves;
    hipLaunchKernelGGL(attn_part_kernel<D>, dim3((unsigned)blocks), dim3(64 * lp.waves), lds, stream, a, lp, po, pm);
    const hipError_t r = hipGetLastError();
    if (r != hipSuccess) return r;
  }
  if (lp.direct) return hipSuccess;
  const bool shared = p.rows_all <= 512;
  const int64_t blocks = shared ? p.rows_all : (p.rows_all + 3) / 4;
  const auto join = shared                ? attn_join_kernel<D, 4>
                    : p.rows_all <= 4096 ? attn_join_kernel<D, 1>
                                          : attn_join_kernel<D, 0>;
  hipLaunchKernelGGL(join, dim3((unsigned)blocks), dim3(256), 0, stream, a, p.rows, p.parts, po, pm);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_prefix(const AttnArgs &a, void *ws, hipStream_t stream) {
  Plan p = plan_for(a);
  p.launch.c = a.scale == 0.f ? 1.f : __builtin_fabsf(a.scale) * ATTN_LOG2E;
  p.launch.qxor = a.scale < 0.f ? 0x80008000u : 0u;
  p.launch.zero = a.scale == 0.f;
  float *po = static_cast<float *>(ws);
  float2 *pm = reinterpret_cast<float2 *>(po + (size_t)p.parts * p.rows_all * a.kv.d);
  return a.kv.d == 64 ? launch_d<64>(a, p, po, pm, stream) : launch_d<128>(a, p, po, pm, stream);
}

}  // namespace oq
