// int8 activations x int8 weights on the gfx950 int8 MFMA (oq_gemm_w8a8).
//
//   y[t][o] = bf16( a_scale[t] w_scale[o] acc[t][o] + mean[t] w1[o] + bias[o] )
//   acc = exact int32 sum over K, converted to float32 with one rounding (a
//   sum of at most 2^31 keeps 24 bits, far more than the bfloat16 output).
//
// Both operands are row-major with K contiguous.  Two kernels:
//
// gemm_w8a8_tile: a workgroup of WM x WN wavefronts, each TI x TJ tiles of
// 32 x 32 on v_mfma_i32_32x32x32_i8, accumulated in place (nothing happens
// between k steps, so the accumulators stay where the MFMA wants them).  k
// advances in stages of 64 through a ring of NSLOT LDS slots, filled global ->
// LDS with 16 rows x 64 bytes per instruction; the 16-byte pieces of a row are
// permuted by the row (on the source side, LDS destinations being linear) so
// that the fragment reads of 16 consecutive rows fall into different banks.
// One barrier per stage; the fragments of the next 32 k are read under the
// MFMAs of the current ones.
#include "oq_internal.h"

#include <cstdlib>

namespace oq {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// what k past the end of the rows is copied from
__device__ const uint4 g_zero16 = {0u, 0u, 0u, 0u};

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

template <int TI_, int TJ_, int WM_, int WN_, int NSLOT_>
struct Tile {
  static constexpr int TI = TI_, TJ = TJ_, WM = WM_, WN = WN_, NSLOT = NSLOT_;
  static constexpr int NW = WM * WN, BM = 32 * TI * WM, BN = 32 * TJ * WN;
  static constexpr int STAGE = (BM + BN) * 64;
  static constexpr int PER = STAGE / 1024 / NW;  // copies per wavefront and stage
  static constexpr int SROW = 64 * TJ + 16;      // bytes of a staged output row of 32 TJ bf16, padded
  static constexpr int LDS = NSLOT * STAGE > NW * 32 * SROW ? NSLOT * STAGE : NW * 32 * SROW;
  static_assert(PER * NW * 1024 == STAGE, "every wavefront copies the same share");
  static_assert(NSLOT == 4, "the waits count for four slots");
  static_assert(LDS <= 160 * 1024, "LDS");
};

template <class C>
__global__ void __launch_bounds__(64 * C::NW, 1) gemm_w8a8_tile(const GemmArgs g) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  constexpr int TI = C::TI, TJ = C::TJ;
  const uint32_t lds0 = lds_addr_of(smem);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, half = lane >> 5;

  // Tile order: workgroups go to the 8 XCDs in turn, each XCD takes a run of
  // tiles, and a run walks column by column through bands of 8 tile rows, so
  // that the 32 tiles an XCD has in flight share rows and columns in its L2.
  const int mt = (int)((g.M + C::BM - 1) / C::BM), nt = (g.N + C::BN - 1) / C::BN;
  const int tiles = mt * nt, xcd = blockIdx.x & 7;
  const int run = tiles >> 3, rem = tiles & 7;
  int id = xcd * run + (xcd < rem ? xcd : rem) + (blockIdx.x >> 3);
  const int band = id / (8 * nt);
  const int bm = mt - 8 * band < 8 ? mt - 8 * band : 8;
  id -= band * 8 * nt;
  const int64_t m0 = (int64_t)(8 * band + id % bm) * C::BM;
  const int n0 = id / bm * C::BN;

  // this wavefront's copies: unit u = wave + NW q covers rows 16 u + lane / 4
  // of the stage (the tile's BM activation rows, then its BN weight rows),
  // 1 KiB at 1024 u of the slot; rows past the end re-read the last one
  const int8_t *src[C::PER];
  int koff[C::PER];
#pragma unroll
  for (int q = 0; q < C::PER; ++q) {
    const int row = 16 * (wave + C::NW * q) + (lane >> 2);
    koff[q] = 16 * ((lane & 3) ^ ((row >> 2) & 3));
    if (row < C::BM) {
      const int64_t m = m0 + row < g.M ? m0 + row : g.M - 1;
      src[q] = g.qa + m * g.lda + koff[q];
    } else {
      const int64_t n = n0 + row - C::BM < g.N ? n0 + row - C::BM : g.N - 1;
      src[q] = g.w + n * g.ldw + koff[q];
    }
  }
  const int S = (g.K + 63) / 64;
  auto issue = [&](int st) {
    const uint32_t base = lds0 + (st & 3) * C::STAGE + 1024 * wave;
    if (64 * st + 64 <= g.K) {
#pragma unroll
      for (int q = 0; q < C::PER; ++q) dma_lds16(src[q] + (int64_t)64 * st, base + 1024 * C::NW * q);
    } else {
#pragma unroll
      for (int q = 0; q < C::PER; ++q)
        dma_lds16(64 * st + koff[q] < g.K ? (const void *)(src[q] + (int64_t)64 * st) : (const void *)&g_zero16,
                  base + 1024 * C::NW * q);
    }
  };

  const int wm = wave / C::WN, wn = wave % C::WN;
  v16i acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = (v16i){};

  // fragment of 32 rows, k 32 kc + 16 half of the stage: row r of the block,
  // piece 2 kc + half in the row's order
  const uint8_t *fa = smem + (wm * 32 * TI + r) * 64, *fb = smem + (C::BM + wn * 32 * TJ + r) * 64;
  const int sw = (r >> 2) & 3;  // (row >> 2) & 3 of every row that is r modulo 32
  auto load = [&](v4i (&a)[TI], v4i (&b)[TJ], int slot, int kc) {
    const int at = slot * C::STAGE + 16 * ((2 * kc + half) ^ sw);
#pragma unroll
    for (int i = 0; i < TI; ++i) a[i] = *reinterpret_cast<const v4i *>(fa + at + i * 2048);
#pragma unroll
    for (int j = 0; j < TJ; ++j) b[j] = *reinterpret_cast<const v4i *>(fb + at + j * 2048);
  };
  auto mma = [&](const v4i (&a)[TI], const v4i (&b)[TJ]) {
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[i], b[j], acc[i][j], 0, 0, 0);
  };

  // Stage s starts with its first fragments in registers.  It waits for this
  // wavefront's copies of stage s + 1 and for its LDS reads; after the barrier
  // stage s + 1 is visible everywhere and nobody reads the slot of stage s - 1
  // any more, which stage s + 3 then fills.
#pragma unroll
  for (int p = 0; p < 3; ++p)
    if (p < S) issue(p);
  if (S > 2) wait_vm<2 * C::PER>();
  else if (S > 1) wait_vm<C::PER>();
  else wait_vm<0>();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  v4i a[2][TI], b[2][TJ];
  load(a[0], b[0], 0, 0);
  for (int s = 0; s < S; ++s) {
    if (s + 2 < S) wait_vm<C::PER>();
    else wait_vm<0>();
    wait_lgkm0();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (s + 3 < S) issue(s + 3);
    __builtin_amdgcn_sched_barrier(0);
    load(a[1], b[1], s & 3, 1);
    mma(a[0], b[0]);
    // after the last stage this reads a slot whose contents are never used
    load(a[0], b[0], (s + 1) & 3, 0);
    mma(a[1], b[1]);
  }

  // Epilogue: 32-row slabs staged in this wavefront's own part of LDS (free
  // once everybody has passed the barrier) for 16-byte stores.
  __syncthreads();
  float ws[TJ], w1v[TJ], bv[TJ];
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    const int col = n0 + 32 * (wn * TJ + j) + r;
    ws[j] = w1v[j] = bv[j] = 0.f;
    if (col < g.N) {
      ws[j] = g.w_scale[col];
      if (g.mean) w1v[j] = g.w1[col];
      if (g.bias) bv[j] = g.bias[col];
    }
  }
  uint8_t *stg = smem + wave * (32 * C::SROW);
  const bool vec_ok = (reinterpret_cast<uintptr_t>(g.y) & 15) == 0 && g.ldy % 8 == 0;
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int64_t mrow = m0 + 32 * (wm * TI + i);
    if (mrow >= g.M) break;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int rr = 8 * (e >> 2) + 4 * half + (e & 3);
      const int64_t row = mrow + rr < g.M ? mrow + rr : g.M - 1;
      const float al = g.a_scale[row], mu = g.mean ? g.mean[row] : 0.f;
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        float v = al * ws[j] * (float)acc[i][j][e];
        if (g.mean) v = __builtin_fmaf(mu, w1v[j], v);
        if (g.bias) v = v + bv[j];
        *reinterpret_cast<uint16_t *>(stg + rr * C::SROW + (32 * j + r) * 2) = f32_to_bf16_rne(v);
      }
    }
    constexpr int CPR = 4 * TJ;  // 16-byte pieces of a slab row
#pragma unroll
    for (int q = 0; q < 2 * TJ; ++q) {
      const int piece = lane + 64 * q;
      const int rr = piece / CPR, cl = (piece % CPR) * 8;
      const int col = n0 + 32 * wn * TJ + cl;
      const u32x4 v = *reinterpret_cast<const u32x4 *>(stg + rr * C::SROW + cl * 2);
      if (mrow + rr >= g.M) continue;
      uint16_t *dst = g.y + (mrow + rr) * g.ldy + col;
      if (vec_ok && col + 8 <= g.N) {
        *reinterpret_cast<u32x4 *>(dst) = v;
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (col + c < g.N) dst[c] = (uint16_t)(v[c >> 1] >> (16 * (c & 1)));
      }
    }
  }
}

// Up to 16 MT rows: a workgroup takes 16 NT weight rows, its NW wavefronts
// the k blocks of 64 in turn, fragments straight from memory (each weight
// byte is used once, so LDS would only add a trip), DEPTH blocks of loads in
// flight per wavefront; the wavefronts' int32 sums meet in LDS.
template <int MT, int NT, int NW, int DEPTH>
__global__ void __launch_bounds__(64 * NW) gemm_w8a8_rows(const GemmArgs g) {
  __shared__ int part[NW][MT * NT * 256];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, kq = 16 * (lane >> 4);
  const int n0 = blockIdx.x * 16 * NT;
  const int8_t *wp[NT], *ap[MT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t n = n0 + 16 * j + r16 < g.N ? n0 + 16 * j + r16 : g.N - 1;
    wp[j] = g.w + n * g.ldw;
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t m = 16 * i + r16 < g.M ? 16 * i + r16 : g.M - 1;
    ap[i] = g.qa + m * g.lda;
  }
  v4i acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = (v4i){};

  const int blocks = (g.K + 63) / 64;
  for (int b0 = wave; b0 < blocks; b0 += NW * DEPTH) {
    v4i W[DEPTH][NT], A[DEPTH][MT];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      // blocks past the end and the missing k of the last one: weights of zero
      const int k = 64 * (b0 + NW * d) + kq;
      const bool ok = k < g.K;
      const int kc = ok ? k : 0;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        W[d][j] = *reinterpret_cast<const v4i *>(wp[j] + kc);
        if (!ok) W[d][j] = (v4i){};
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) A[d][i] = *reinterpret_cast<const v4i *>(ap[i] + kc);
    }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(A[d][i], W[d][j], acc[i][j], 0, 0, 0);
  }
  // lane: column (weight row) l % 16, rows 4 (l / 16) + e
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[wave][(i * NT + j) * 256 + (4 * (lane >> 4) + e) * 16 + r16] = acc[i][j][e];
  __syncthreads();
  for (int at = threadIdx.x; at < MT * NT * 256; at += 64 * NW) {
    const int blk = at / 256, i = blk / NT, j = blk % NT;
    const int64_t row = 16 * i + (at % 256) / 16;
    const int col = n0 + 16 * j + at % 16;
    if (row >= g.M || col >= g.N) continue;
    int s = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) s += part[w][at];
    float v = g.a_scale[row] * g.w_scale[col] * (float)s;
    if (g.mean) v = __builtin_fmaf(g.mean[row], g.w1[col], v);
    if (g.bias) v = v + g.bias[col];
    g.y[row * g.ldy + col] = f32_to_bf16_rne(v);
  }
}

template <class C>
hipError_t launch_tile(const GemmArgs &g, hipStream_t stream) {
  static std::atomic<bool> attr_set[64];
  const hipError_t e = lds_limit_once((const void *)gemm_w8a8_tile<C>, C::LDS, attr_set);
  if (e != hipSuccess) return e;
  const int64_t tiles = ((g.M + C::BM - 1) / C::BM) * ((g.N + C::BN - 1) / C::BN);
  if (tiles > 0x7fffffff) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(gemm_w8a8_tile<C>, dim3((unsigned)tiles), dim3(64 * C::NW), C::LDS, stream, g);
  return hipGetLastError();
}

template <int MT, int NT, int NW, int DEPTH>
hipError_t launch_rows(const GemmArgs &g, hipStream_t stream) {
  hipLaunchKernelGGL((gemm_w8a8_rows<MT, NT, NW, DEPTH>), dim3((unsigned)((g.N + 16 * NT - 1) / (16 * NT))), dim3(64 * NW), 0,
                     stream, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_w8a8(const int8_t *qa, int64_t lda, const float *a_scale, int64_t M, int32_t K, const int8_t *w,
                            int64_t ldw, const float *w_scale, int N, const float *mean, const float *w1,
                            const float *bias, uint16_t *y, int64_t ldy, hipStream_t stream) {
  const GemmArgs g{qa, lda, a_scale, M, K, w, ldw, w_scale, N, mean, w1, bias, y, ldy};
  int f = 0;
  if (const char *e = getenv("W8")) f = atoi(e);
  if (f == 1 && M <= 16) return launch_rows<1, 1, 4, 8>(g, stream);
  if (f == 2 && M <= 32) return launch_rows<2, 1, 4, 8>(g, stream);
  if (f == 3) return launch_tile<Tile<1, 1, 2, 2, 4>>(g, stream);
  if (f == 4) return launch_tile<Tile<2, 2, 2, 2, 4>>(g, stream);
  if (f == 5) return launch_tile<Tile<4, 4, 2, 2, 4>>(g, stream);
  if (f == 6) return launch_tile<Tile<4, 2, 2, 4, 4>>(g, stream);
  if (f == 7 && M <= 16) return launch_rows<1, 1, 8, 8>(g, stream);
  if (f == 8 && M <= 16) return launch_rows<1, 1, 8, 4>(g, stream);
  if (f == 9 && M <= 16) return launch_rows<1, 1, 16, 4>(g, stream);
  if (f == 10 && M <= 16) return launch_rows<1, 1, 4, 16>(g, stream);
  if (f == 11 && M <= 16) return launch_rows<1, 2, 4, 8>(g, stream);
  if (M <= 16) return launch_rows<1, 1, 4, 8>(g, stream);
  if (M <= 32) return launch_rows<2, 1, 4, 8>(g, stream);
  if (((M + 255) / 256) * ((N + 255) / 256) >= 128) return launch_tile<Tile<4, 4, 2, 2, 4>>(g, stream);
  if (((M + 127) / 128) * ((N + 127) / 128) >= 128) return launch_tile<Tile<2, 2, 2, 2, 4>>(g, stream);
  return launch_tile<Tile<1, 1, 2, 2, 4>>(g, stream);
}

}  // namespace oq
