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
// advances in stages of 128 through a ring of NSLOT LDS slots, filled global ->
// LDS with 8 rows x 128 bytes per instruction; the 16-byte pieces of a row are
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
  static constexpr int STAGE = (BM + BN) * 128;
  static constexpr int PER = STAGE / 1024 / NW;  // copies per wavefront and stage
  static constexpr int SROW = 64 * TJ + 16;      // bytes of a staged output row of 32 TJ bf16, padded
  static constexpr int VEC = NSLOT * STAGE > NW * 32 * SROW ? NSLOT * STAGE : NW * 32 * SROW;
  static constexpr int LDS = VEC + 2 * BM * 4;   // the ring or the staged slabs, row scales and means
  static_assert(PER * NW * 1024 == STAGE, "every wavefront copies the same share");
  static_assert(NSLOT >= 2 && (NSLOT - 2) * PER <= 63, "vmcnt range");
  static_assert(LDS <= 160 * 1024, "LDS");
};

template <class C>
__global__ void __launch_bounds__(64 * C::NW, C::NW == 8 || C::LDS <= 80 * 1024 ? 2 : 1) gemm_w8a8_tile(const GemmArgs g) {
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

  // this wavefront's copies: unit u = wave + NW q covers rows 8 u + lane / 8
  // of the stage (the tile's BM activation rows, then its BN weight rows),
  // 1 KiB at 1024 u of the slot; rows past the end re-read the last one
  const int8_t *src[C::PER];
  int koff[C::PER];
#pragma unroll
  for (int q = 0; q < C::PER; ++q) {
    const int row = 8 * (wave + C::NW * q) + (lane >> 3);
    koff[q] = 16 * ((lane & 7) ^ ((row >> 1) & 7));
    if (row < C::BM) {
      const int64_t m = m0 + row < g.M ? m0 + row : g.M - 1;
      src[q] = g.qa + m * g.lda + koff[q];
    } else {
      const int64_t n = n0 + row - C::BM < g.N ? n0 + row - C::BM : g.N - 1;
      src[q] = g.w + n * g.ldw + koff[q];
    }
  }
  const int S = (g.K + 127) / 128;
  // src[] always points at stage `next`: its copies past K (the last stage of
  // a K that is no multiple of 128) and past the last stage come from zeros, so
  // that the loop below has no special stages
  int next = 0, fill = 0;  // that stage and its slot
  auto zero_past = [&](int k) {
#pragma unroll
    for (int q = 0; q < C::PER; ++q)
      if (koff[q] >= k) src[q] = reinterpret_cast<const int8_t *>(&g_zero16);
  };
  if (S == 1) zero_past(g.K);
  auto issue = [&](int q) { dma_lds16(src[q], lds0 + fill * C::STAGE + 1024 * wave + 1024 * C::NW * q); };
  auto advance = [&]() {
    ++next;
    fill = fill == C::NSLOT - 1 ? 0 : fill + 1;
    if (next < S) {
#pragma unroll
      for (int q = 0; q < C::PER; ++q) src[q] += 128;
      if (next == S - 1) zero_past(g.K - 128 * next);
    } else if (next == S) {
      zero_past(0);
    }
  };

  float *s_scale = reinterpret_cast<float *>(smem + C::VEC), *s_mean = s_scale + C::BM;
  for (int t = threadIdx.x; t < C::BM; t += 64 * C::NW) {
    const int64_t row = m0 + t < g.M ? m0 + t : g.M - 1;
    s_scale[t] = g.a_scale[row];
    s_mean[t] = g.mean ? g.mean[row] : 0.f;
  }

  const int wm = wave / C::WN, wn = wave % C::WN;
  v16i acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = (v16i){};

  // fragment of 32 rows, k 32 kc + 16 half of the stage: row r of the block,
  // piece 2 kc + half in the row's order
  const uint8_t *fa = smem + (wm * 32 * TI + r) * 128, *fb = smem + (C::BM + wn * 32 * TJ + r) * 128;
  const int sw = (r >> 1) & 7;  // (row >> 1) & 7 of every row that is r modulo 32

  // One chunk of 32 k: the MFMAs of each row block under the reads of the next
  // chunk's fragments and this wavefront's share of the next copies, spread
  // over the first half of a stage's MFMAs so that neither holds them up.
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
      for (int j = 0; j < TJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[i], b[j], acc[i][j], 0, 0, 0);
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
#pragma unroll
  for (int p = 0; p < C::NSLOT - 1; ++p) {
#pragma unroll
    for (int q = 0; q < C::PER; ++q) issue(q);
    advance();
  }
  int slot = 0;
  for (int s = 0; s < S; ++s) {
    wait_vm<(C::NSLOT - 2) * C::PER>();
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
    for (int j = 0; j < TJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[0][i], b[0][j], acc[i][j], 0, 0, 0);
  wait_vm<0>();  // the slots are reused

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
    for (int e4 = 0; e4 < 4; ++e4) {
      const int r4 = 8 * e4 + 4 * half;  // rows r4 .. r4 + 3 of the slab
      const float4 al4 = *reinterpret_cast<const float4 *>(s_scale + 32 * (wm * TI + i) + r4);
      const float4 mu4 = *reinterpret_cast<const float4 *>(s_mean + 32 * (wm * TI + i) + r4);
      const float al[4] = {al4.x, al4.y, al4.z, al4.w}, mu[4] = {mu4.x, mu4.y, mu4.z, mu4.w};
#pragma unroll
      for (int e1 = 0; e1 < 4; ++e1)
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
          float v = al[e1] * ws[j] * (float)acc[i][j][4 * e4 + e1];
          if (g.mean) v = __builtin_fmaf(mu[e1], w1v[j], v);
          if (g.bias) v = v + bv[j];
          *reinterpret_cast<uint16_t *>(stg + (r4 + e1) * C::SROW + (32 * j + r) * 2) = f32_to_bf16_rne(v);
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
  if (f == 4) return launch_tile<Tile<2, 2, 2, 2, 2>>(g, stream);
  if (f == 5) return launch_tile<Tile<4, 4, 2, 2, 2>>(g, stream);
  if (f == 6) return launch_tile<Tile<4, 2, 2, 4, 2>>(g, stream);
  if (f == 12) return launch_tile<Tile<2, 2, 2, 2, 3>>(g, stream);
  if (f == 13) return launch_tile<Tile<2, 2, 2, 2, 4>>(g, stream);
  if (f == 14) return launch_tile<Tile<2, 4, 4, 2, 2>>(g, stream);
  if (f == 7 && M <= 16) return launch_rows<1, 1, 8, 8>(g, stream);
  if (f == 8 && M <= 16) return launch_rows<1, 1, 8, 4>(g, stream);
  if (f == 9 && M <= 16) return launch_rows<1, 1, 16, 4>(g, stream);
  if (f == 10 && M <= 16) return launch_rows<1, 1, 4, 16>(g, stream);
  if (f == 11 && M <= 16) return launch_rows<1, 2, 4, 8>(g, stream);
  if (M <= 16) return launch_rows<1, 1, 4, 8>(g, stream);
  if (M <= 32) return launch_rows<2, 1, 4, 8>(g, stream);
  if (((M + 255) / 256) * ((N + 255) / 256) >= 128) return launch_tile<Tile<4, 2, 2, 4, 2>>(g, stream);
  if (((M + 127) / 128) * ((N + 127) / 128) >= 128) return launch_tile<Tile<2, 2, 2, 2, 4>>(g, stream);
  return launch_tile<Tile<1, 1, 2, 2, 4>>(g, stream);
}

}  // namespace oq
