// int8 activations x int8 weights on the gfx950 int8 MFMA (oq_gemm_w8a8).
//
//   y[t][o] = bf16( a_scale[t] w_scale[o] acc[t][o] + mean[t] w1[o] + bias[o] )
//   acc = exact int32 sum over K, converted to float32 with one rounding (a
//   sum of at most 2^31 keeps 24 bits, far more than the bfloat16 output).
//
// Both operands are row-major with K contiguous.  Up to 32 tokens the weights
// have to be read and little else, and few outputs need k split to fill the chip:
// gemm_w8a8_rows.  Else gemm_w8a8_tile: a
// workgroup of WM x WN wavefronts, each TI x TJ tiles of
// 32 x 32 on v_mfma_i32_32x32x32_i8, accumulated in place (nothing happens
// between k steps, so the accumulators stay where the MFMA wants them).  k
// advances in stages of 128 through a ring of NSLOT LDS slots, filled global ->
// LDS with 8 rows x 128 bytes per instruction; the 16-byte pieces of a row are
// permuted by the row (on the source side, LDS destinations being linear) so
// that the fragment reads of 16 consecutive rows fall into different banks.
// One barrier per stage; the fragments of the next 32 k are read under the
// MFMAs of the current ones.
//
// What bounds it.  The 256 x 256 tile: the matrix unit at the clock that the
// operands' bits allow, 8192 x 4096 -> 14336 takes 432 to 463 us on one card and
// another, 2.1 to 2.2 POP/s (a large int8 product of the library: 2.16; the
// instruction alone 4.7).  The smaller
// tiles: copies into LDS (64 bytes a clock and CU, so 556 clocks for a stage of
// the 128 x 128 tile against 512 of products) and products overlap to seven
// tenths; 512 x 4096 -> 4096 takes 16.8 us, 333 x 1920 -> 7680 10.4.
#include "oq_internal.h"

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

struct GemmArgs {
  const int8_t *qa;
  int64_t lda;
  const float *a_scale;
  int64_t M;
  int K;
  const int8_t *w;
  int64_t ldw;
  const float *w_scale;
  int N;
  const float *mean, *w1, *bias;
  uint16_t *y;
  int64_t ldy;
};

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

// How workgroups map to tiles.
struct TileMap {
  int mt, nt;      // tile rows and columns
  int run, rem;    // tiles / 8, tiles % 8
  Div band, full, last;  // 8 nt; tile rows of a full band; of the last band
};

template <int TI_, int TJ_, int WM_, int WN_, int NSLOT_>
struct Tile {
  static constexpr int TI = TI_, TJ = TJ_, WM = WM_, WN = WN_, NSLOT = NSLOT_;
  static constexpr int NW = WM * WN, BM = 32 * TI * WM, BN = 32 * TJ * WN;
  static constexpr int STAGE = (BM + BN) * 128;
  static constexpr int PER = STAGE / 1024 / NW;  // copies per wavefront and stage
  // copies NW q .. NW q + NW - 1 are activation rows (weight rows follow them)
  static constexpr bool A_UNIT(int q) { return 8 * NW * q < BM; }
  static constexpr int SROW = 80;                // bytes of a staged row of 32 bf16, padded
  static constexpr int STG = NW * TJ * 32 * SROW, RING = NSLOT * STAGE;
  static constexpr int VEC = RING > STG ? RING : STG, LDS = VEC + 3 * BN * 4;
  static constexpr int RESIDENT = 160 * 1024 / LDS < 4 ? 160 * 1024 / LDS : 4;  // workgroups a CU
  static_assert(PER * NW * 1024 == STAGE, "every wavefront copies the same share");
  static_assert(BM % (8 * NW) == 0 && NW % 2 == 0, "a round of copies is all activations or all weights");
  static_assert(NSLOT >= 2 && (NSLOT - 2) * PER <= 63, "vmcnt range");
  static_assert(BN <= 64 * NW, "one thread per column");
  static_assert(LDS <= 160 * 1024, "LDS");
};

template <class C>
__global__ void __launch_bounds__(64 * C::NW, C::NW / 4 * C::RESIDENT) gemm_w8a8_tile(const GemmArgs g, const TileMap t) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  constexpr int TI = C::TI, TJ = C::TJ;
  const uint32_t lds0 = lds_addr_of(smem);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, half = lane >> 5;

  // Tile order: workgroups go to the 8 XCDs in turn; each XCD takes a run of
  // tiles, and a run walks column by column through bands of 8 tile rows, so
  // that the tiles that an XCD has in flight share rows and columns in its L2.
  const int xcd = blockIdx.x & 7;
  const int id = xcd * t.run + (xcd < t.rem ? xcd : t.rem) + (blockIdx.x >> 3);
  const int band = div_of(id, t.band), in_band = id - band * t.band.d;
  const Div rows = 8 * band + 8 <= t.mt ? t.full : t.last;
  const int tn = div_of(in_band, rows);
  const int64_t m0 = (int64_t)(8 * band + in_band - tn * rows.d) * C::BM;
  const int n0 = tn * C::BN;

  // This wavefront's copies: unit u = wave + NW q covers rows 8 u + lane / 8
  // of the stage (the tile's BM activation rows, then its BN weight rows),
  // 1 KiB at 1024 u of the slot; rows past the end re-read the last one.
  // base_a, base_w (scalar) point at stage `next`, voff[] is each lane's place
  // below them, slot `fill` takes the stage.
  const int S = (g.K + 127) / 128, last_k = g.K - 128 * (S - 1);  // k of the last stage
  int next = 0, fill = 0;
  uint32_t voff[C::PER];
  const int piece = 16 * ((lane & 7) ^ ((lane >> 4) | (wave & 1) << 2));  // of its row: every row of a lane has this (row >> 1) & 7
  const int8_t *base_a = g.qa + m0 * g.lda, *base_w = g.w + (int64_t)n0 * g.ldw;
  {
    const int ma = g.M - m0 < C::BM ? (int)(g.M - m0) - 1 : C::BM - 1, na = g.N - n0 < C::BN ? g.N - n0 - 1 : C::BN - 1;
#pragma unroll
    for (int q = 0; q < C::PER; ++q) {
      const int row = 8 * (wave + C::NW * q) + (lane >> 3);
      if (C::A_UNIT(q)) voff[q] = (uint32_t)(row < ma ? row : ma) * (uint32_t)g.lda + piece;
      else voff[q] = (uint32_t)(row - C::BM < na ? row - C::BM : na) * (uint32_t)g.ldw + piece;
    }
  }
  auto issue = [&](int q) {
    dma_lds16_s(C::A_UNIT(q) ? base_a : base_w, voff[q], lds0 + fill * C::STAGE + 1024 * wave + 1024 * C::NW * q);
  };
  // what lies past K in the last stage is copied from the row's first piece of
  // the stage and cleared in LDS (clear_tail)
  auto tail_offsets = [&]() {
    if (piece < last_k) return;
#pragma unroll
    for (int q = 0; q < C::PER; ++q) voff[q] -= piece;
  };
  if (S == 1) tail_offsets();
  // After the last stage the loop goes on copying 16 bytes of it all over slots
  // that nobody reads, so that it has no special stages.
  auto advance = [&]() {
    ++next;
    fill = fill == C::NSLOT - 1 ? 0 : fill + 1;
    if (next < S) {
      base_a += 128;
      base_w += 128;
      if (next == S - 1) tail_offsets();
    } else if (next == S) {
#pragma unroll
      for (int q = 0; q < C::PER; ++q) voff[q] = 0;
    }
  };
  auto clear_tail = [&](int slot) {  // activations past K become zeros, each wavefront clearing what it copied
    if (piece < last_k) return;
#pragma unroll
    for (int q = 0; q < C::PER; ++q)
      if (C::A_UNIT(q))
        *reinterpret_cast<v4i *>(smem + slot * C::STAGE + 1024 * (wave + C::NW * q) + 16 * lane) = (v4i){};
  };
#pragma unroll
  for (int p = 0; p < C::NSLOT - 1; ++p) {
#pragma unroll
    for (int q = 0; q < C::PER; ++q) issue(q);
    advance();
  }

  // the epilogue's vectors, used after the main loop
  const int wm = wave / C::WN, wn = wave % C::WN;
  float ws = 0.f, w1 = 0.f, bias = 0.f, al[TI], mu[TI];
  {
    const int col = n0 + (int)threadIdx.x;
    if (threadIdx.x < C::BN && col < g.N) {
      ws = g.w_scale[col];
      if (g.mean) w1 = g.w1[col];
      if (g.bias) bias = g.bias[col];
    }
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int64_t row = m0 + 32 * (wm * TI + i) + r < g.M ? m0 + 32 * (wm * TI + i) + r : g.M - 1;
      al[i] = g.a_scale[row];
      mu[i] = g.mean ? g.mean[row] : 0.f;
    }
  }

  // fragment of 32 rows, k 32 kc + 16 half of the stage: row r of the block,
  // piece 2 kc + half in the row's order
  const uint8_t *fa = smem + (wm * 32 * TI + r) * 128, *fb = smem + (C::BM + wn * 32 * TJ + r) * 128;
  const int sw = (r >> 1) & 7;  // (row >> 1) & 7 of every row that is r modulo 32

  v16i acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = (v16i){};
  // One chunk of 32 k: the MFMAs of each row block under the reads of the next
  // chunk's fragments and this wavefront's share of the next copies, spread
  // over the first half of a stage's MFMAs so that neither holds them up.  The
  // product is formed transposed (rows: weights), so that a lane holds one
  // token and four consecutive outputs per group of four registers.
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

  // The loop is turned by one chunk: when the last chunk of stage s - 1 is in
  // registers, nobody needs its slot any more.  So there the wavefronts wait
  // for their copies of stage s, meet, run that chunk while the fragments of
  // stage s come in, and send the copies of stage s + NSLOT - 1 to the slot.
  v4i a[2][TI], b[2][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i) a[0][i] = (v4i){};  // the chunk before stage 0
#pragma unroll
  for (int j = 0; j < TJ; ++j) b[0][j] = (v4i){};
  int slot = 0;
  for (int s = 0; s < S; ++s) {
    wait_vm<(C::NSLOT - 2) * C::PER>();
    asm volatile("" ::: "memory");
    if (s == S - 1 && last_k < 128) clear_tail(slot);
    wait_lgkm0();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
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

  // Epilogue, in the ring's place once nobody copies to or reads from it: each
  // wavefront stages the TJ tiles of a row block for 16-byte stores.  Without
  // a mean or bias their zeros are added.
  float *s_ws = reinterpret_cast<float *>(smem + C::VEC), *s_w1 = s_ws + C::BN, *s_b = s_w1 + C::BN;
  if (threadIdx.x < C::BN) {
    s_ws[threadIdx.x] = ws;
    s_w1[threadIdx.x] = w1;
    s_b[threadIdx.x] = bias;
  }
  wait_vm<0>();
  asm volatile("" ::: "memory");
  __syncthreads();
  uint8_t *stg = smem + wave * (TJ * 32 * C::SROW);
  const bool vec_ok = (reinterpret_cast<uintptr_t>(g.y) & 15) == 0 && g.ldy % 8 == 0;
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int64_t mrow = m0 + 32 * (wm * TI + i);
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {
        const int c = 32 * (wn * TJ + j) + 8 * e4 + 4 * half;
        const float4 s4 = *reinterpret_cast<const float4 *>(s_ws + c);
        const float4 w4 = *reinterpret_cast<const float4 *>(s_w1 + c);
        const float4 b4 = *reinterpret_cast<const float4 *>(s_b + c);
        const float v0 = __builtin_fmaf(mu[i], w4.x, al[i] * s4.x * (float)acc[i][j][4 * e4]) + b4.x;
        const float v1 = __builtin_fmaf(mu[i], w4.y, al[i] * s4.y * (float)acc[i][j][4 * e4 + 1]) + b4.y;
        const float v2 = __builtin_fmaf(mu[i], w4.z, al[i] * s4.z * (float)acc[i][j][4 * e4 + 2]) + b4.z;
        const float v3 = __builtin_fmaf(mu[i], w4.w, al[i] * s4.w * (float)acc[i][j][4 * e4 + 3]) + b4.w;
        *reinterpret_cast<uint2 *>(stg + (32 * j + r) * C::SROW + 16 * e4 + 8 * half) =
            make_uint2((uint32_t)f32_to_bf16_rne(v0) | ((uint32_t)f32_to_bf16_rne(v1) << 16),
                       (uint32_t)f32_to_bf16_rne(v2) | ((uint32_t)f32_to_bf16_rne(v3) << 16));
      }
    }
#pragma unroll
    for (int q = 0; q < 2 * TJ; ++q) {
      const int at = (lane >> 2) + 16 * q;  // staged row: 32 per tile
      const int64_t row = mrow + (at & 31);
      const int col = n0 + 32 * (wn * TJ + (at >> 5)) + 8 * (lane & 3);
      const u32x4 v = *reinterpret_cast<const u32x4 *>(stg + at * C::SROW + 16 * (lane & 3));
      if (row >= g.M) continue;
      uint16_t *dst = g.y + row * g.ldy + col;
      if (vec_ok && col + 8 <= g.N) {
        *reinterpret_cast<u32x4 *>(dst) = v;
      } else {
        for (int x = 0; x < 8 && col + x < g.N; ++x) dst[x] = (uint16_t)(v[x >> 1] >> (16 * (x & 1)));
      }
    }
  }
}

// 16 MT tokens (a group of them: blockIdx.y) times 16 weight rows a workgroup, its
// 8 wavefronts the k blocks of 64 in turn.  Weight fragments come straight from memory (each byte
// is used once, so LDS would only add a trip), two batches of 2 loads in flight
// per wavefront; the activations, which every workgroup reads, go through LDS in
// chunks of as many k as fit, sent before the first weight loads and with each
// row's 16-byte pieces permuted by the row against bank conflicts.  The
// wavefronts' int32 sums meet in LDS.  Measured: 1 x 4096 x 6144 7.8 us (batches
// of 4 7.8, of 8 11), 16 x 1920 x 7680 5.8 (7.3, 10.8), 32 x 4096 x 14336 19.8
// (3.0 TB/s of weights).  A chunk's copies and first weights start when the last
// one has been used, and the epilogue's vectors are asked for after the sums have
// met: both are trips to memory that nothing hides.
template <int MT>
__global__ void __launch_bounds__(512) gemm_w8a8_rows(const GemmArgs g, const int CH) {
  constexpr int NW = 8, DEPTH = 2;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  __shared__ int part[NW][MT * 256];
  const uint32_t lds0 = lds_addr_of(smem);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, kq = lane >> 4;
  const int64_t n = (int64_t)blockIdx.x * 16 + r16;
  const int8_t *wp = g.w + (n < g.N ? n : g.N - 1) * g.ldw + 16 * kq;
  const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
  const int8_t *qa = g.qa + m0 * g.lda;
  const int rows = g.M - m0 < 16 * MT ? (int)(g.M - m0) : 16 * MT;
  v4i acc[MT];
  const uint8_t *arow[MT];  // rows past M are not stored
  int asw[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    acc[i] = (v4i){};
    const int row = 16 * i + r16 < rows ? 16 * i + r16 : rows - 1;
    arow[i] = smem + row * CH;
    asw[i] = row & 15;
  }
  for (int k0 = 0; k0 < g.K; k0 += CH) {
    const int kn = g.K - k0 < CH ? g.K - k0 : CH, blocks = (kn + 63) / 64;
    // weights of blocks b, b + NW, ..; what lies past the chunk is zero
    auto load = [&](v4i (&W)[DEPTH], int b) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        const int k = 64 * (b + NW * d);
        W[d] = *reinterpret_cast<const v4i *>(wp + (k + 16 * kq < kn ? k0 + k : -16 * kq));
      }
    };
    auto use = [&](v4i (&W)[DEPTH], int b) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        const int blk = b + NW * d;
        if (blk >= blocks) break;
        if (64 * blk + 16 * kq >= kn) W[d] = (v4i){};
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const v4i A = *reinterpret_cast<const v4i *>(arow[i] + 16 * ((4 * blk + kq) ^ asw[i]));
          acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(A, W[d], acc[i], 0, 0, 0);
        }
      }
    };
    // 1 KiB pieces of the chunk's activations, rows in turn
    const int per_row = CH / 1024;
    for (int u = wave; u < rows * per_row; u += NW) {
      const int row = u / per_row, k = 1024 * (u - row * per_row) + 16 * (lane ^ (row & 15));
      dma_lds16(qa + row * g.lda + (k < kn ? k0 + k : 0), lds0 + 1024 * u);
    }
    asm volatile("" ::: "memory");
    v4i W[2][DEPTH];
    load(W[0], wave);
    load(W[1], wave + NW * DEPTH);
    asm volatile("" ::: "memory");
    wait_vm<2 * DEPTH>();  // the activations; the weights may still come
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    for (int b = wave; b < blocks; b += 2 * NW * DEPTH) {
      use(W[0], b);
      if (b + 2 * NW * DEPTH < blocks) load(W[0], b + 2 * NW * DEPTH);
      use(W[1], b + NW * DEPTH);
      if (b + 3 * NW * DEPTH < blocks) load(W[1], b + 3 * NW * DEPTH);
    }
    wait_vm<0>();  // weights past the chunk that nobody used: else the next copies wait for each other
    if (k0 + CH < g.K) __syncthreads();
  }
  // lane: column (weight row) l % 16, rows 4 (l / 16) + e
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) part[wave][i * 256 + (4 * kq + e) * 16 + r16] = acc[i][e];
  __syncthreads();
  const int at = threadIdx.x;
  const int64_t row = m0 + at / 16, col = (int64_t)blockIdx.x * 16 + at % 16;
  if (at >= MT * 256 || row >= g.M || col >= g.N) return;
  int s = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) s += part[w][at];
  // as in the tiles, zeros stand for what is not given: the sign of a zero too
  // does not depend on the kernel
  const float v = g.a_scale[row] * g.w_scale[col] * (float)s;
  const float r = __builtin_fmaf(g.mean ? g.mean[row] : 0.f, g.mean ? g.w1[col] : 0.f, v);
  g.y[row * g.ldy + col] = f32_to_bf16_rne(r + (g.bias ? g.bias[col] : 0.f));
}

template <class C>
hipError_t launch_tile(const GemmArgs &g, hipStream_t stream) {
  static std::atomic<bool> attr_set[64];
  const hipError_t e = lds_limit_once((const void *)gemm_w8a8_tile<C>, C::LDS, attr_set);
  if (e != hipSuccess) return e;
  const int64_t mt = (g.M + C::BM - 1) / C::BM, nt = (g.N + C::BN - 1) / C::BN;
  if (mt * nt > 0x7fffffff || 8 * nt > 0x7fffffff) return hipErrorInvalidConfiguration;
  const int tiles = (int)(mt * nt);
  const TileMap t{(int)mt, (int)nt, tiles / 8, tiles % 8, div_by((uint32_t)(8 * nt)), div_by(8), div_by(mt % 8 ? (uint32_t)(mt % 8) : 8)};
  hipLaunchKernelGGL(gemm_w8a8_tile<C>, dim3((unsigned)tiles), dim3(64 * C::NW), C::LDS, stream, g, t);
  return hipGetLastError();
}

template <int MT>
hipError_t launch_rows(const GemmArgs &g, hipStream_t stream) {
  // 64 KiB of activations at a time lets two workgroups share a CU; where one
  // round of workgroups covers N, 128 KiB.  16 tokens, K = 14336, N = 4096: 16.6
  // us with 128 KiB against 17.5; 32 tokens, K = N = 4096: 8.9 against 9.5
  // (both before the wait at the chunk's end, 14.9 and 7.9 since).
  const int64_t nt = (g.N + 15) / 16, mt = (g.M + 16 * MT - 1) / (16 * MT);
  const int lds = nt * mt <= device_cus() ? 131072 : 65536;
  const int rows = g.M < 16 * MT ? (int)g.M : 16 * MT;
  int ch = lds / 1024 / rows * 1024;
  if (ch > (g.K + 1023) / 1024 * 1024) ch = (g.K + 1023) / 1024 * 1024;
  static std::atomic<bool> attr_set[64];
  const hipError_t e = lds_limit_once((const void *)gemm_w8a8_rows<MT>, 131072, attr_set);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(gemm_w8a8_rows<MT>, dim3((unsigned)nt, (unsigned)mt), dim3(512), (size_t)rows * ch, stream, g, ch);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_w8a8(const int8_t *qa, int64_t lda, const float *a_scale, int64_t M, int32_t K, const int8_t *w,
                            int64_t ldw, const float *w_scale, int N, const float *mean, const float *w1,
                            const float *bias, uint16_t *y, int64_t ldy, hipStream_t stream) {
  const GemmArgs g{qa, lda, a_scale, M, K, w, ldw, w_scale, N, mean, w1, bias, y, ldy};
  // Eight wavefronts on the k of 16 x 16 outputs, where those tiles are no more
  // than the CUs: 100 x 14336 x 500 13.4 us (64 x 64 tiles, whose few workgroups
  // would each walk all of k: 30), 64 x 4096 x 64 5.3 (10.4), 32 x 14336 x 2048
  // 14.0 (32 x 16 outputs: 18.7).
  const int64_t cus = device_cus(), nt = ((int64_t)N + 15) / 16;
  if (M <= 16 || nt * ((M + 15) / 16) <= cus) return launch_rows<1>(g, stream);
  if (M <= 32) return launch_rows<2>(g, stream);
  // The tile with the least modelled time, rounds of workgroups over the CUs
  // times the measured time of a round at K = 4096 (us): 256 x 256 59, 128 x 256
  // 34, 128 x 128 22, 64 x 64 7.3 and 4 for the first.  K scales a round, not the
  // fixed part of a call, so the choice is the measured one at K = 4096 and is
  // taken for every K.
  // Measured with K = 4096, N = 4096: 512 tokens 42.7 / 25.6 / 19.4 / 16.3, 1024
  // 44.2 / 28.5 / 22.1 / 30, 2048 47.4 / 36.2 / 40.6, 4096 63.4 / 67.4 / 77.4;
  // 1952 x 13984 x 8705 419 / 396 / 431 / 613.
  // Against them gemm_w8a8_rows<2>, 2.8 and 4 for a round of 32 x 16 outputs a CU:
  // 128 tokens, N = 1024 6.8 (64 x 64 tiles 10.9), N = 2048 10.6 (11.1).
  auto rounds = [&](int64_t bm, int64_t bn) { return (double)(((M + bm - 1) / bm * ((N + bn - 1) / bn) + cus - 1) / cus); };
  const double c256 = 59 * rounds(256, 256), c384 = 34 * rounds(128, 256), c128 = 22 * rounds(128, 128),
               c64 = 4 + 7.3 * rounds(64, 64), c512 = 2.8 + 4 * rounds(32, 16);
  if (c512 <= c64 && c512 <= c128) return launch_rows<2>(g, stream);
  if (c256 <= c384 && c256 <= c128 && c256 <= c64) return launch_tile<Tile<2, 4, 4, 2, 2>>(g, stream);
  if (c384 <= c128 && c384 <= c64) return launch_tile<Tile<2, 2, 2, 4, 3>>(g, stream);
  if (c128 <= c64) return launch_tile<Tile<2, 1, 2, 4, 3>>(g, stream);
  return launch_tile<Tile<1, 1, 2, 2, 3>>(g, stream);
}

}  // namespace oq
