// The experts' int8 products (oq_gemm_w8a8_experts): every entry's activation
// row times the weights of its expert, on the gfx950 int8 MFMA.
//
//   v[i][o] = a_scale w_scale[e] acc + mean w1[e] + bias[e],  acc exact in int32
//   y[i][o] = bf16(v)   or   bf16(silu(v[gate]) v[up])
//
// The host does not know how many entries an expert has: a wavefront finds its
// tile's expert from the E offsets by a sum across its lanes, and tiles that are
// not there end at once.  An entry's activation row is found through the list when
// it is copied into LDS, and its output goes to the entry's own row, so nothing is
// gathered or sorted in memory.  With SwiGLU a wavefront's two blocks of weight rows
// are a gate's and the same outputs' up rows: both sums are in the same lane and
// registers, and the projections' 2 f values never exist.
//
// What bounds it.  Few entries an expert: the weights, read once, at copy rate
// (16 x 8 entries of 128 experts, 2048 -> 1536: 41 to 47 us, 260 MB; a copy of as
// many bytes takes 50).  Many: the matrix unit at the clock that power allows, a stage
// of 128 k of a 128 x 256 tile a CU in 1.0 us (2.15 POP/s; the library's largest int8
// product reaches 2.4), and what is not product: 3 us between two tiles, 1.2 us of
// epilogue, 2 us of stores, a sixteenth to an eighth of the rows empty in the experts' last
// tiles.  8192 x 8 entries of 128 experts, 2048 -> 1536: 274 to 302 us of 172 for the
// products alone at the library's rate; 4096 k, 64 experts: 465 of 344; 768 -> 2048: 207 of 100.
// Outputs that 16-byte stores do not fit (N or ldy no multiple of 8) go two bytes at a time.
#include "sparse_plan.h"

namespace oq {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <int C>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt(0x0F70 | (C & 0xF) | ((C >> 4) << 14));
}

__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(0xC07F); }

// x / d for a divisor whose reciprocal r = floor(2^32 / d) + 1 the host has
// formed: the high product is the quotient or one more.
struct Div {
  uint32_t d, r;
};
__host__ inline Div div_by(uint32_t d) { return {d, d == 1 ? 0u : (uint32_t)((1ull << 32) / d + 1)}; }
__device__ __forceinline__ uint32_t div_of(uint32_t x, Div v) {
  if (v.d == 1) return x;
  const uint32_t q = __umulhi(x, v.r);
  return q * v.d > x ? q - 1 : q;
}

// Entries order[p0] .. order[p0 + rows - 1] of expert e, against column tile tn;
// rows 0: no such tile.
struct Place {
  int e, p0, rows, tn;
};

// An address that all lanes share, in scalar registers.
__device__ __forceinline__ const int8_t *scalar(const int8_t *p) {
  const uint64_t a = (uint64_t)p;
  return (const int8_t *)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(a >> 32)) << 32 |
                          (uint32_t)__builtin_amdgcn_readfirstlane((int)a));
}

// Row tiles of the lanes up to and with this one, of which it has `tiles`.  Lists as
// oq_route makes them have no more than n / TM + E; of others the sum stays in 32
// bits all the same (n <= 2^28).
template <int TM>
__device__ __forceinline__ int tiles_below(const ExpertArgs &g, int tiles) {
  const int lane = threadIdx.x & 63, most = (int)g.n / TM + g.E;
  int sum = tiles > most ? most : tiles;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(sum, o);
    if (lane >= o) sum += u;
  }
  return sum;
}

// Tiles of an XCD's run: an eighth of them (2^28 at most, so that places in all runs have 32 bits;
// the grid's size says that those of oq_route's lists are fewer).
__device__ __forceinline__ int run_of(int rows, int nt) {
  const int64_t run = ((int64_t)rows * nt + 7) / 8;
  return run < 1 << 28 ? (int)run : 1 << 28;
}

// Tile of this workgroup, `block` of all launches, TM entries a row tile, nt column tiles.
// Workgroups go to the 8 XCDs in turn; each XCD takes a run of tiles, the columns of a row tile one
// after the other, so that what it has in flight are the tiles of one expert or two,
// whose rows and weights its L2 holds.  The same in every lane.
template <int TM>
__device__ __forceinline__ Place find_tile(const ExpertArgs &g, int nt, uint32_t block) {
  const int lane = threadIdx.x & 63, n = (int)g.n, each = (g.E + 63) / 64;
  auto cut = [&](int v) { return v < 0 ? 0 : v < n ? v : n; };
  const int e0 = lane * each, e1 = e0 + each < g.E ? e0 + each : g.E;
  int tiles = 0;  // 16 experts of 2^28 entries at most
  if (e0 < e1) {
    int at = cut(g.offsets[e0]);
    for (int e = e0; e < e1; ++e) {
      const int next = cut(g.offsets[e + 1]);
      tiles += next > at ? (next - at + TM - 1) / TM : 0;
      at = next;
    }
  }
  const int sum = tiles_below<TM>(g, tiles);  // up to and with this lane
  Place r{0, 0, 0, 0};
  const int rows = __builtin_amdgcn_readlane(sum, 63), run = run_of(rows, nt);
  const int in_run = block >> 3, id = (block & 7) * run + in_run;
  const int tile = __builtin_amdgcn_readfirstlane((int)((uint32_t)id / (uint32_t)nt));
  if (in_run >= run || tile >= rows) return r;
  r.tn = id - tile * nt;
  const int win = __ffsll((long long)__ballot(sum > tile)) - 1;
  int left = tile - __builtin_amdgcn_readlane(sum - tiles, win);
  const int f0 = win * each, f1 = f0 + each < g.E ? f0 + each : g.E;
  int at = cut(g.offsets[f0]);
  for (int e = f0; e < f1; ++e) {
    const int next = cut(g.offsets[e + 1]), here = next > at ? (next - at + TM - 1) / TM : 0;
    if (left < here) {
      r.e = e;
      r.p0 = at + left * TM;
      r.rows = next - r.p0 < TM ? next - r.p0 : TM;
      break;
    }
    left -= here;
    at = next;
  }
  return r;
}

// v = silu(v) up.  The exponential of v log2(e) and the reciprocal are the instructions',
// good to some 2^-22 (1 + |v|), far below the bfloat16 result, while the denominator and its
// reciprocal are normal numbers: down to v = -87.  Below -80 it is v e^v up, which can be
// far above e^v: with h = e^(v / 2), a normal number down to v = -174, (v h) up h; then 0.
// (With this form for all negative v 8192 x 8 entries take another 3 to 5 us.)
template <int N>
__device__ __forceinline__ void silu_mul(float (&v)[N], const float (&up)[N]) {
  constexpr float LOG2E = 1.44269504088896340736f, FAR = -80.f;
  float y[N], least = v[0];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    y[i] = v[i] * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v[i] * -LOG2E)) * up[i];
    least = fminf(least, v[i]);
  }
  if (__any(least < FAR)) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float h = __builtin_amdgcn_exp2f(v[i] * (0.5f * LOG2E));
      y[i] = v[i] < FAR ? v[i] * h * up[i] * h : y[i];
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = y[i];
}

// Up to 16 MT entries times 32 (8 / KS) weight rows a workgroup: wavefront w takes
// weight rows of block w / KS and the k blocks of 128 that are w % KS modulo KS.
// Weights come straight from memory, each byte being used once: a lane's two
// loads of a block are 32 bytes in a row, four lanes a line of 128 (the order of k
// within a block does not matter to the sum, as long as the activations have the
// same).  The activations, which every wavefront reads, go through LDS in chunks
// of CH bytes, each row's 16-byte pieces permuted by the row against bank
// conflicts.
template <int MT, int KS, bool ACT>
__global__ void __launch_bounds__(512) gemm_experts_rows(const ExpertArgs g, const uint32_t first, const int CH, const int nt, const Div per) {
  constexpr int NW = 8, TM = 16 * MT, GROUPS = NW / KS, DEPTH = 2;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Place rt = find_tile<TM>(g, nt, first + blockIdx.x);
  if (rt.rows == 0) return;
  const uint32_t lds0 = lds_addr_of(smem);
  const int r16 = lane & 15, kq = lane >> 4, ks = wave % KS;
  const int half = ACT ? g.N / 2 : g.N;
  const int n0 = (rt.tn * GROUPS + wave / KS) * (ACT ? 16 : 32);  // first output of this wavefront
  // weight rows of this lane's column in both blocks; rows past the end re-read the last one
  const int c0 = n0 + r16, c1 = ACT ? c0 : c0 + 16;
  const int q0 = c0 < half ? c0 : half - 1, q1 = ACT ? half + q0 : c1 < half ? c1 : half - 1;
  const int8_t *w = g.w + rt.e * g.w_stride + 32 * kq;
  const int8_t *w0 = w + q0 * g.ldw, *w1 = w + q1 * g.ldw;
  auto entry = [&](int r) {  // of row r of the tile; -1: none
    const int i = g.order[rt.p0 + r];
    return i >= 0 && i < g.n ? i : -1;
  };

  v4i acc[MT][2];
  const uint8_t *arow[MT];  // rows past the tile's are not stored
  int asw[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    acc[i][0] = acc[i][1] = (v4i){};
    const int row = 16 * i + r16 < rt.rows ? 16 * i + r16 : rt.rows - 1;
    arow[i] = smem + row * CH;
    asw[i] = row & 15;
  }
  for (int k0 = 0; k0 < g.K; k0 += CH) {
    const int kn = g.K - k0 < CH ? g.K - k0 : CH, blocks = (kn + 127) / 128;
    // block b of both weight rows; what lies past the chunk is zero
    auto load = [&](v4i (&W)[4], int b) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = 128 * b + 16 * h, at = k + 32 * kq < kn ? k0 + k : -32 * kq;
        W[h] = *reinterpret_cast<const v4i *>(w0 + at);
        W[2 + h] = *reinterpret_cast<const v4i *>(w1 + at);
      }
    };
    auto use = [&](v4i (&W)[4], int b) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (128 * b + 16 * h + 32 * kq >= kn) W[h] = W[2 + h] = (v4i){};
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const v4i A = *reinterpret_cast<const v4i *>(arow[i] + 16 * ((8 * b + 2 * kq + h) ^ asw[i]));
          acc[i][0] = __builtin_amdgcn_mfma_i32_16x16x64_i8(A, W[h], acc[i][0], 0, 0, 0);
          acc[i][1] = __builtin_amdgcn_mfma_i32_16x16x64_i8(A, W[2 + h], acc[i][1], 0, 0, 0);
        }
      }
    };
    // 1 KiB pieces of the chunk's activations, rows in turn
    const int per_row = CH / 1024;
    for (int u = wave; u < rt.rows * per_row; u += NW) {
      const int row = u / per_row, k = 1024 * (u - row * per_row) + 16 * (lane ^ (row & 15));
      const int i = entry(row);
      dma_lds16(g.qa + (int64_t)(i < 0 ? 0 : div_of(i, per)) * g.lda + (k < kn ? k0 + k : 0), lds0 + 1024 * u);
    }
    v4i W[DEPTH][4];
#pragma unroll
    for (int p = 0; p < DEPTH; ++p) load(W[p], ks + KS * p);
    wait_vm<0>();
    asm volatile("" ::: "memory");
    __syncthreads();
    for (int b = ks; b < blocks; b += DEPTH * KS) {
#pragma unroll
      for (int p = 0; p < DEPTH; ++p) {
        if (b + KS * p >= blocks) break;
        use(W[p], b + KS * p);
        load(W[p], b + KS * (p + DEPTH));
      }
    }
    __syncthreads();
  }

  // lane: weight row r16 of each block, entries 4 kq + x
  if (KS > 1) {  // the wavefronts' sums of k meet, in the activations' place
    int *part = reinterpret_cast<int *>(smem);
    if (ks > 0) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int b = 0; b < 2; ++b) *reinterpret_cast<v4i *>(part + ((wave * MT + i) * 2 + b) * 256 + 4 * lane) = acc[i][b];
    }
    __syncthreads();
    if (ks > 0) return;
#pragma unroll
    for (int s = 1; s < KS; ++s)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int b = 0; b < 2; ++b) acc[i][b] += *reinterpret_cast<const v4i *>(part + (((wave + s) * MT + i) * 2 + b) * 256 + 4 * lane);
  }
  const int64_t at = (int64_t)rt.e * g.N;
  const float s0 = g.w_scale[at + q0], s1 = g.w_scale[at + q1];
  const float m0 = g.mean ? g.w1[at + q0] : 0.f, m1 = g.mean ? g.w1[at + q1] : 0.f;
  const float b0 = g.bias ? g.bias[at + q0] : 0.f, b1 = g.bias ? g.bias[at + q1] : 0.f;
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int row = 16 * i + 4 * kq + x;
      if (row >= rt.rows) continue;
      const int en = entry(row);
      if (en < 0) continue;
      const uint32_t from = div_of(en, per);
      const float as = g.a_scale[from], mu = g.mean ? g.mean[from] : 0.f;
      float v0[1] = {__builtin_fmaf(mu, m0, as * s0 * (float)acc[i][0][x]) + b0};
      const float v1[1] = {__builtin_fmaf(mu, m1, as * s1 * (float)acc[i][1][x]) + b1};
      uint16_t *y = g.y + en * g.ldy;
      if (ACT) {
        silu_mul(v0, v1);
        if (c0 < half) y[c0] = f32_to_bf16_rne(v0[0]);
      } else {
        if (c0 < half) y[c0] = f32_to_bf16_rne(v0[0]);
        if (c1 < half) y[c1] = f32_to_bf16_rne(v1[0]);
      }
    }
}

// Tiles of BM entries x BN weight rows: WM x WN wavefronts, each TI x TJ blocks of 32 x 32 on
// v_mfma_i32_32x32x32_i8, k in stages of 128 through a ring of NSLOT LDS slots.
template <int TI_, int TJ_, int WM_, int WN_, int NSLOT_>
struct Tile {
  static constexpr int TI = TI_, TJ = TJ_, WM = WM_, WN = WN_, NSLOT = NSLOT_;
  static constexpr int NW = WM * WN, BM = 32 * TI * WM, BN = 32 * TJ * WN;
  static constexpr int STAGE = (BM + BN) * 128;
  static constexpr int PER = STAGE / 1024 / NW;  // copies per wavefront and stage
  static constexpr int PER_A = BM / 8 / NW;      // of which the first are activation rows
  static constexpr int RING = NSLOT * STAGE;
  // behind the ring: w_scale, w1, bias of the columns, a_scale, mean of the rows, the rows' entries of
  // this tile and the next, the experts' first places and tiles (MAX_E + 1 and MAX_E of them)
  static constexpr int MAX_E = 1024;
  static constexpr int AT_ROWS = RING + 3 * BN * 4, AT_ENTRY = AT_ROWS + 2 * BM * 4, AT_LISTS = AT_ENTRY + 2 * BM * 4;
  static constexpr int LDS = AT_LISTS + (2 * MAX_E + 1) * 4;
  static constexpr int MIN_STAGES = NSLOT + 1;  // of a tile: the next one's entries are there before its first copies
  static_assert(PER * NW * 1024 == STAGE, "every wavefront copies the same share");
  static_assert(BM % (8 * NW) == 0 && NW % 4 == 0, "a round of copies is all activations or all weights");
  static_assert(NSLOT == 3, "vectors sent behind a stage's barrier are older than all that the next one leaves open");
  static_assert(BN <= 64 * NW && BM <= 64 * NW, "one thread per column and row");
  static_assert(TJ % 2 == 0, "gate and up blocks of a wavefront in turn");
  static_assert(LDS <= 160 * 1024, "LDS");
};

// A persistent kernel, one workgroup a CU: the ring does not end with a tile.  Under
// the last stages of one the first stages of the next one are copied, and what else
// the next one needs (its entries, scales) comes through LDS as well, so that its
// main loop starts at full pace.  Where a workgroup took one tile, 8192 x 8 entries
// of 128 experts, 2048 -> 1536, took 313 us: 8 of a tile's 23 us passed before its
// first product and behind its last.
template <class C, bool ACT>
__global__ void __launch_bounds__(64 * C::NW, C::NW / 4) gemm_experts_tile(const ExpertArgs g, const int nt, const Div per) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  constexpr int TI = C::TI, TJ = C::TJ, OUT = ACT ? C::BN / 2 : C::BN;
  const uint32_t lds0 = lds_addr_of(smem);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, half = lane >> 5;
  const int outs = ACT ? g.N / 2 : g.N;
  float *s_ws = reinterpret_cast<float *>(smem + C::RING), *s_w1 = s_ws + C::BN, *s_b = s_w1 + C::BN;
  float *s_al = reinterpret_cast<float *>(smem + C::AT_ROWS), *s_mu = s_al + C::BM;
  int *s_entry = reinterpret_cast<int *>(smem + C::AT_ENTRY);  // [2][BM]
  int *s_off = reinterpret_cast<int *>(smem + C::AT_LISTS), *s_sum = s_off + C::MAX_E + 1;

  // the experts' first places, and the tiles up to and with each of them
  const int each = (g.E + 63) / 64;
  if (wave == 0) {
    const int n = (int)g.n;
    auto cut = [&](int v) { return v < 0 ? 0 : v < n ? v : n; };
    for (int e = lane; e <= g.E; e += 64) s_off[e] = cut(g.offsets[e]);
    const int e0 = lane * each, e1 = e0 + each < g.E ? e0 + each : g.E;
    int tiles = 0;  // 16 experts of 2^28 entries at most
    for (int e = e0; e < e1; ++e) {
      const int rows = s_off[e + 1] - s_off[e];
      tiles += rows > 0 ? (rows + C::BM - 1) / C::BM : 0;
      s_sum[e] = tiles;
    }
    const int below = tiles_below<C::BM>(g, tiles) - tiles;
    for (int e = e0; e < e1; ++e) s_sum[e] += below;
  }
  // what is not given is zero
  for (int i = threadIdx.x; i < 2 * C::BN; i += 64 * C::NW) s_w1[i] = 0.f;
  for (int i = threadIdx.x; i < C::BM; i += 64 * C::NW) s_mu[i] = 0.f;
  __syncthreads();
  const int tiles = __builtin_amdgcn_readfirstlane(s_sum[g.E - 1]), run = __builtin_amdgcn_readfirstlane(run_of(tiles, nt));
  // Tile `it` of this workgroup: as at find_tile an XCD takes a run of tiles, here those of an expert in
  // bands of 8 row tiles, column by column, so that many columns share rows and weights as well
  // (8192 rows of one expert, 4096 -> 14336: 509 us; row by row 590).
  auto find = [&](int it) {
    Place p{0, 0, 0, 0};
    const int in_run = (blockIdx.x >> 3) + it * (gridDim.x >> 3), id = (blockIdx.x & 7) * run + in_run;
    const int tile = __builtin_amdgcn_readfirstlane((int)((uint32_t)id / (uint32_t)nt));
    if (in_run >= run || tile >= tiles) return p;
    const int last = lane * each + each - 1;
    const uint64_t past = __ballot(s_sum[last < g.E ? last : g.E - 1] > tile);
    const int first = (__ffsll((long long)past) - 1) * each, mine = first + (lane < each ? lane : each - 1);
    const uint64_t in = __ballot(s_sum[mine < g.E ? mine : g.E - 1] > tile);
    p.e = __builtin_amdgcn_readfirstlane(first + __ffsll((long long)in) - 1);
    const int before = __builtin_amdgcn_readfirstlane(p.e ? s_sum[p.e - 1] : 0), own = __builtin_amdgcn_readfirstlane(s_sum[p.e]) - before;
    const int start = __builtin_amdgcn_readfirstlane(s_off[p.e]), end = __builtin_amdgcn_readfirstlane(s_off[p.e + 1]);
    // bands of 8 row tiles, column by column
    const uint32_t local = (uint32_t)(id - before * nt), wide = 8 * (uint32_t)nt;
    const uint32_t band = __builtin_amdgcn_readfirstlane((int)(local / wide)), in_band = local - band * wide;
    const uint32_t high = own - 8 * (int)band < 8 ? own - 8 * (int)band : 8;
    p.tn = __builtin_amdgcn_readfirstlane((int)(in_band / (high ? high : 1)));
    const int64_t at = start + ((int64_t)8 * band + in_band - p.tn * high) * C::BM;
    if (at < start || at >= end || p.tn >= nt) return p;  // not with oq_route's lists
    p.p0 = (int)at;
    p.rows = end - p.p0 < C::BM ? end - p.p0 : C::BM;
    return p;
  };
  Place rt = find(0), nx = rt;
  if (rt.rows <= 0) return;
  auto checked = [&](int i) { return i >= 0 && i < g.n ? i : -1; };  // an entry from a list; -1: none
  auto entry = [&](const Place &p, const int *list, int row) { return row < p.rows ? checked(list[row]) : -1; };
  auto from = [&](int i) { return (int64_t)(i < 0 ? 0 : div_of(i, per)); };
  // weight row of column c of the tile (with SwiGLU its blocks of 32 are gate and up rows in turn),
  // relative to the first gate or up row; past the end the last one
  auto weight_row = [&](const Place &p, int c) {
    const int o = ACT ? (c >> 6) * 32 + (c & 31) : c, last = outs - p.tn * OUT - 1;
    return o < last ? o : last;
  };
  auto is_up = [&](int c) { return ACT && (c >> 5 & 1); };

  // This wavefront's copies: unit u = wave + NW q covers rows 8 u + lane / 8 of the
  // stage (the tile's BM activation rows, then its BN weight rows), 1 KiB at 1024 u
  // of the slot.  Activation rows have addresses of their own, weight rows an offset
  // below a scalar base.  Slot `fill` takes stage `next` of the tile.
  const int S = (g.K + 127) / 128, last_k = g.K - 128 * (S - 1);  // k of the last stage
  int next = 0, fill = 0;
  const int piece = 16 * ((lane & 7) ^ ((lane >> 4) | (wave & 1) << 2));  // of its row: every row of a lane has this (row >> 1) & 7
  const int8_t *arow[C::PER_A], *base_w, *base_up;
  uint32_t voff[C::PER - C::PER_A];
  auto aim = [&](const Place &p, const int *list) {
    base_w = g.w + p.e * g.w_stride + (int64_t)p.tn * OUT * g.ldw;
    base_up = base_w + (ACT ? (int64_t)outs * g.ldw : 0);
#pragma unroll
    for (int q = 0; q < C::PER; ++q) {
      const int row = 8 * (wave + C::NW * q) + (lane >> 3);
      if (q < C::PER_A) arow[q] = g.qa + from(entry(p, list, row)) * g.lda + piece;
      else voff[q - C::PER_A] = (uint32_t)weight_row(p, row - C::BM) * (uint32_t)g.ldw + piece;
    }
  };
  const int8_t *now_w, *now_up;  // the bases of the stage whose copies are being sent
  auto settle = [&]() { now_w = scalar(base_w), now_up = scalar(base_up); };
  auto issue = [&](int q) {
    const uint32_t to = lds0 + fill * C::STAGE + 1024 * wave + 1024 * C::NW * q;
    if (q < C::PER_A) dma_lds16(arow[q], to);
    else dma_lds16_s(is_up(8 * (wave + C::NW * q) - C::BM) ? now_up : now_w, voff[q - C::PER_A], to);
  };
  // what lies past K in the last stage is copied from the row's first piece of
  // the stage and cleared in LDS (clear_tail)
  auto tail_offsets = [&]() {
    if (piece < last_k) return;
#pragma unroll
    for (int q = 0; q < C::PER_A; ++q) arow[q] -= piece;
#pragma unroll
    for (int q = C::PER_A; q < C::PER; ++q) voff[q - C::PER_A] -= piece;
  };
  // Behind the last stage of the last tile the loop goes on copying 16 bytes all
  // over slots that nobody reads, so that it has no special stages.
  int flip = 0;  // which entries are this tile's
  auto advance = [&]() {
    ++next;
    fill = fill == C::NSLOT - 1 ? 0 : fill + 1;
    if (next < S) {
#pragma unroll
      for (int q = 0; q < C::PER_A; ++q) arow[q] += 128;
      base_w += 128;
      base_up += 128;
      if (next == S - 1) tail_offsets();
    } else if (next == S) {
      if (nx.rows > 0) {
        aim(nx, s_entry + (flip ^ 1) * C::BM);
        next = 0;
      } else {
#pragma unroll
        for (int q = 0; q < C::PER_A; ++q) arow[q] = base_w;
#pragma unroll
        for (int q = C::PER_A; q < C::PER; ++q) voff[q - C::PER_A] = 0;
      }
    }
  };
  auto clear_tail = [&](int slot) {  // activations past K become zeros, each wavefront clearing what it copied
    if (piece < last_k) return;
#pragma unroll
    for (int q = 0; q < C::PER_A; ++q)
      *reinterpret_cast<v4i *>(smem + slot * C::STAGE + 1024 * (wave + C::NW * q) + 16 * lane) = (v4i){};
  };
  // A tile's vectors and the next one's entries, sent once every wavefront is done with the last
  // tile's and read a barrier later.  64 columns or rows a wavefront at a time.
  auto send_vectors = [&]() {
    for (int u = wave; u < C::BN / 64; u += C::NW) {
      const int c = 64 * u + lane;
      const int64_t at = (int64_t)rt.e * g.N + rt.tn * OUT + weight_row(rt, c) + (is_up(c) ? outs : 0);
      dma_lds4(g.w_scale + at, lds0 + C::RING + 256 * u);
      if (g.mean) dma_lds4(g.w1 + at, lds0 + C::RING + 4 * C::BN + 256 * u);
      if (g.bias) dma_lds4(g.bias + at, lds0 + C::RING + 8 * C::BN + 256 * u);
    }
    for (int u = C::NW - 1 - wave; u < C::BM / 64; u += C::NW) {
      const int row = 64 * u + lane;
      const int64_t at = from(entry(rt, s_entry + flip * C::BM, row));
      dma_lds4(g.a_scale + at, lds0 + C::AT_ROWS + 256 * u);
      if (g.mean) dma_lds4(g.mean + at, lds0 + C::AT_ROWS + 4 * C::BM + 256 * u);
      if (nx.rows > 0)
        dma_lds4(g.order + nx.p0 + (row < nx.rows ? row : nx.rows - 1), lds0 + C::AT_ENTRY + (flip ^ 1) * C::BM * 4 + 256 * u);
    }
  };

  if (threadIdx.x < C::BM) s_entry[threadIdx.x] = threadIdx.x < rt.rows ? g.order[rt.p0 + threadIdx.x] : -1;
  __syncthreads();
  aim(rt, s_entry);
#pragma unroll
  for (int p = 0; p < C::NSLOT - 1; ++p) {
    settle();
#pragma unroll
    for (int q = 0; q < C::PER; ++q) issue(q);
    advance();  // not to another tile: MIN_STAGES
  }

  // fragment of 32 rows, k 32 kc + 16 half of the stage: row r of the block,
  // piece 2 kc + half in the row's order
  const int wm = wave / C::WN, wn = wave % C::WN;
  const uint8_t *fa = smem + (wm * 32 * TI + r) * 128, *fb = smem + (C::BM + wn * 32 * TJ + r) * 128;
  const int sw = (r >> 1) & 7;  // (row >> 1) & 7 of every row that is r modulo 32
  v16i acc[TI][TJ];
  // One chunk of 32 k: the MFMAs of each row block under the reads of the next
  // chunk's fragments and this wavefront's share of the next copies, spread over
  // the first half of a stage's MFMAs.  The product is formed transposed (rows:
  // weights), so that a lane holds one entry and four outputs in a row.
  constexpr int GROUPS = 2 * TI;
  auto chunk = [&](const v4i (&a)[TI], const v4i (&b)[TJ], v4i (&an)[TI], v4i (&bn)[TJ], int slot, int kc, int part) {
    const int at = slot * C::STAGE + 16 * ((2 * kc + half) ^ sw);
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      an[i] = *reinterpret_cast<const v4i *>(fa + at + i * 4096);
#pragma unroll
      for (int j = i * TJ / TI; j < (i + 1) * TJ / TI; ++j) bn[j] = *reinterpret_cast<const v4i *>(fb + at + j * 4096);
      if (part < 2) {
#pragma unroll
        for (int q = (part * TI + i) * C::PER / GROUPS; q < (part * TI + i + 1) * C::PER / GROUPS; ++q) issue(q);
      }
#pragma unroll
      for (int j = 0; j < TJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b[j], a[i], acc[i][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  const bool vec_ok = (reinterpret_cast<uintptr_t>(g.y) & 15) == 0 && g.ldy % 8 == 0;
  constexpr int BLOCKS = ACT ? TJ / 2 : TJ;  // of 32 outputs a wavefront
  int slot = 0;
  for (int it = 1;; ++it) {
    nx = find(it);
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j) acc[i][j] = (v16i){};
    // The loop is turned by one chunk: when the last chunk of stage s - 1 is in
    // registers, nobody needs its slot any more.  So there the wavefronts wait for
    // their copies of stage s, meet, run that chunk while the fragments of stage s
    // come in, and send the copies of stage s + NSLOT - 1 to the slot.
    v4i a[2][TI], b[2][TJ];
#pragma unroll
    for (int i = 0; i < TI; ++i) a[0][i] = (v4i){};  // the chunk before stage 0
#pragma unroll
    for (int j = 0; j < TJ; ++j) b[0][j] = (v4i){};
    for (int s = 0; s < S; ++s) {
      if (s > 0 || it == 1) wait_vm<(C::NSLOT - 2) * C::PER>();
      asm volatile("" ::: "memory");
      if (s == S - 1 && last_k < 128) clear_tail(slot);
      wait_lgkm0();
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      settle();
      if (s == 0) send_vectors();  // older than the stage's copies: there when the next barrier opens
      chunk(a[0], b[0], a[1], b[1], slot, 0, 0);
      chunk(a[1], b[1], a[0], b[0], slot, 1, 1);
      advance();
      chunk(a[0], b[0], a[1], b[1], slot, 2, 2);
      chunk(a[1], b[1], a[0], b[0], slot, 3, 3);
      slot = slot == C::NSLOT - 1 ? 0 : slot + 1;
    }
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(b[0][j], a[0][i], acc[i][j], 0, 0, 0);

    // the next tile's first stage, before stores that would have to be waited for with it
    wait_vm<(C::NSLOT - 2) * C::PER>();
    asm volatile("" ::: "memory");
    // Epilogue, straight from the registers: of the four outputs that a lane has of
    // every eight, the wavefront's halves exchange two fours, so that each stores 16
    // bytes in a row.  Without a mean or bias their zeros are added.
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int row = 32 * (wm * TI + i) + r;
      const int en = entry(rt, s_entry + flip * C::BM, row);
      const float al = s_al[row], mu = s_mu[row];
      auto values = [&](int j, int e4, float (&v)[4]) {
        const int c = 32 * (wn * TJ + j) + 8 * e4 + 4 * half;
        const float4 s4 = *reinterpret_cast<const float4 *>(s_ws + c);
        const float4 w4 = *reinterpret_cast<const float4 *>(s_w1 + c);
        const float4 b4 = *reinterpret_cast<const float4 *>(s_b + c);
        v[0] = __builtin_fmaf(mu, w4.x, al * s4.x * (float)acc[i][j][4 * e4]) + b4.x;
        v[1] = __builtin_fmaf(mu, w4.y, al * s4.y * (float)acc[i][j][4 * e4 + 1]) + b4.y;
        v[2] = __builtin_fmaf(mu, w4.z, al * s4.z * (float)acc[i][j][4 * e4 + 2]) + b4.z;
        v[3] = __builtin_fmaf(mu, w4.w, al * s4.w * (float)acc[i][j][4 * e4 + 3]) + b4.w;
      };
#pragma unroll
      for (int k = 0; k < BLOCKS; ++k) {
#pragma unroll
        for (int e8 = 0; e8 < 2; ++e8) {
          uint32_t w[2][2];  // outputs 8 (2 e8 + x) + 4 half ..
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float v[4];
            if constexpr (ACT) {
              float up[4];
              values(2 * k, 2 * e8 + x, v);
              values(2 * k + 1, 2 * e8 + x, up);
              silu_mul(v, up);
            } else {
              values(k, 2 * e8 + x, v);
            }
            w[x][0] = (uint32_t)f32_to_bf16_rne(v[0]) | ((uint32_t)f32_to_bf16_rne(v[1]) << 16);
            w[x][1] = (uint32_t)f32_to_bf16_rne(v[2]) | ((uint32_t)f32_to_bf16_rne(v[3]) << 16);
          }
          u32x4 o;
#pragma unroll
          for (int y = 0; y < 2; ++y) {  // lower lanes: outputs 16 e8 .. + 7, upper lanes the next eight
            const auto sw2 = __builtin_amdgcn_permlane32_swap(w[0][y], w[1][y], false, false);
            o[y] = sw2[0];
            o[2 + y] = sw2[1];
          }
          const int col = rt.tn * OUT + 32 * (wn * BLOCKS + k) + 16 * e8 + 8 * half;
          uint16_t *dst = g.y + en * g.ldy + col;
          if (en < 0) continue;
          if (vec_ok && col + 8 <= outs) {
            *reinterpret_cast<u32x4 *>(dst) = o;
          } else {
            for (int y = 0; y < 8 && col + y < outs; ++y) dst[y] = (uint16_t)(o[y >> 1] >> (16 * (y & 1)));
          }
        }
      }
    }
    if (nx.rows <= 0) break;
    rt = nx;
    flip ^= 1;
  }
  wait_vm<0>();  // copies into LDS that nobody waited for
}

// Tiles need more than NSLOT stages.
template <class C, bool ACT>
hipError_t launch_tile(const ExpertArgs &g, const ExpertPlan &p, hipStream_t stream) {
  static_assert(C::BM == EXPERT_BM && C::BN == EXPERT_BN && C::MIN_STAGES == EXPERT_STAGES, "the plan's tiles");
  static std::atomic<bool> attr_set[64];
  const hipError_t e = lds_limit_once((const void *)gemm_experts_tile<C, ACT>, C::LDS, attr_set);
  if (e != hipSuccess) return e;
  const int64_t cus = device_cus() < 8 ? 8 : device_cus() / 8 * 8, grid = p.grid < cus ? p.grid : cus;
  hipLaunchKernelGGL((gemm_experts_tile<C, ACT>), dim3((unsigned)grid), dim3(64 * C::NW), C::LDS, stream, g, (int)p.columns,
                     div_by((uint32_t)g.per));
  return hipGetLastError();
}

template <int MT, int KS, bool ACT>
hipError_t launch_rows(const ExpertArgs &g, const ExpertPlan &p, hipStream_t stream) {
  constexpr int TM = 16 * MT, PART = 8 * MT * 2 * 1024;
  int ch = 65536 / TM / 1024 * 1024;
  if (ch > (g.K + 1023) / 1024 * 1024) ch = (g.K + 1023) / 1024 * 1024;
  const size_t lds = (size_t)TM * ch > PART || KS == 1 ? (size_t)TM * ch : PART;
  constexpr int64_t MOST = rows_of_launch(512) / 8 * 8;  // workgroups, whole turns of the XCDs
  for (int64_t first = 0; first < p.grid; first += MOST) {
    hipLaunchKernelGGL((gemm_experts_rows<MT, KS, ACT>), dim3((unsigned)(p.grid - first < MOST ? p.grid - first : MOST)), dim3(512), lds, stream, g,
                       (uint32_t)first, ch, (int)p.columns, div_by((uint32_t)g.per));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool ACT>
hipError_t launch(const ExpertArgs &g, hipStream_t stream) {
  const ExpertPlan p = expert_plan(g.n, g.K, g.N, g.E, ACT);
  if (p.grid > 0x7fffffff) return hipErrorInvalidConfiguration;
  if (p.mt == 0) return launch_tile<Tile<2, 2, 2, 4, 3>, ACT>(g, p, stream);
  if (p.mt == 4) return launch_rows<4, 1, ACT>(g, p, stream);
  if (p.ks == 8) return launch_rows<1, 8, ACT>(g, p, stream);
  if (p.ks == 4) return launch_rows<1, 4, ACT>(g, p, stream);
  if (p.ks == 2) return launch_rows<1, 2, ACT>(g, p, stream);
  return launch_rows<1, 1, ACT>(g, p, stream);
}

}  // namespace

hipError_t launch_gemm_experts(const ExpertArgs &g, int act, hipStream_t stream) {
  return act == OQ_ACT_SWIGLU ? launch<true>(g, stream) : launch<false>(g, stream);
}

}  // namespace oq
