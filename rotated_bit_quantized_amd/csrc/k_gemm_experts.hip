// The experts' int8 products (oq_gemm_w8a8_experts): every entry's activation
// row times the weights of its expert, on the gfx950 int8 MFMA.
//
//   v[i][o] = a_scale w_scale[e] acc + mean w1[e] + bias[e],  acc exact in int32
//   y[i][o] = bf16(v)   or   bf16(silu(v[gate]) v[up])
//
// The host does not know how many entries an expert has.  The grid covers the
// most row tiles that n entries of E experts can make, n / TM + min(E, n); every
// wavefront finds its tile's expert from the E offsets by a cross-lane sum, and
// tiles that are not there end at once.  An entry's row is found through the
// list when it is copied into LDS, and its output goes to the entry's own row,
// so nothing is gathered or sorted in memory.  With SwiGLU a wavefront's two
// blocks of weight rows are a gate's and the same outputs' up rows: both sums
// are in the same lane and registers, and the intermediate never exists.
#include "oq_internal.h"

namespace oq {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

template <int C>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt(0x0F70 | (C & 0xF) | ((C >> 4) << 14));
}

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

// Entries order[p0] .. order[p0 + rows - 1] of expert e; rows 0: no such tile.
struct RowTile {
  int e, p0, rows;
};

// Row tile `tile` of the lists, TM entries a tile.  The same in every lane.
template <int TM>
__device__ __forceinline__ RowTile find_tile(const ExpertArgs &g, int tile) {
  const int lane = threadIdx.x & 63, n = (int)g.n, each = (g.E + 63) / 64;
  auto cut = [&](int v) { return v < 0 ? 0 : v < n ? v : n; };
  const int e0 = lane * each, e1 = e0 + each < g.E ? e0 + each : g.E;
  int tiles = 0;
  if (e0 < e1) {
    int at = cut(g.offsets[e0]);
    for (int e = e0; e < e1; ++e) {
      const int next = cut(g.offsets[e + 1]);
      tiles += next > at ? (next - at + TM - 1) / TM : 0;
      at = next;
    }
  }
  int sum = tiles;  // up to and with this lane
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(sum, o);
    if (lane >= o) sum += u;
  }
  const uint64_t past = __ballot(sum > tile);
  RowTile r{0, 0, 0};
  if (past == 0) return r;
  const int win = __ffsll((long long)past) - 1;
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

__device__ __forceinline__ float silu_mul(float gate, float up) { return gate / (1.f + expf(-gate)) * up; }

// Up to 16 MT entries times 32 (8 / KS) weight rows a workgroup: wavefront w takes
// weight rows of block w / KS and the k blocks of 128 that are w % KS modulo KS.
// Weights come straight from memory, each byte being used once: a lane's two
// loads of a block are 32 bytes in a row, four lanes a line of 128 (the order of k
// within a block does not matter to the sum, as long as the activations have the
// same).  The activations, which every wavefront reads, go through LDS in chunks
// of CH bytes, each row's 16-byte pieces permuted by the row against bank
// conflicts.
template <int MT, int KS, bool ACT>
__global__ void __launch_bounds__(512) gemm_experts_rows(const ExpertArgs g, const int CH, const int nt, const Div per) {
  constexpr int NW = 8, TM = 16 * MT, GROUPS = NW / KS, DEPTH = 2;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tile = blockIdx.x / nt, tn = blockIdx.x - tile * nt;
  const RowTile rt = find_tile<TM>(g, tile);
  if (rt.rows == 0) return;
  const uint32_t lds0 = lds_addr_of(smem);
  const int r16 = lane & 15, kq = lane >> 4, ks = wave % KS;
  const int half = ACT ? g.N / 2 : g.N;
  const int n0 = (tn * GROUPS + wave / KS) * (ACT ? 16 : 32);  // first output of this wavefront
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
      const float v0 = __builtin_fmaf(mu, m0, as * s0 * (float)acc[i][0][x]) + b0;
      const float v1 = __builtin_fmaf(mu, m1, as * s1 * (float)acc[i][1][x]) + b1;
      uint16_t *y = g.y + en * g.ldy;
      if (ACT) {
        if (c0 < half) y[c0] = f32_to_bf16_rne(silu_mul(v0, v1));
      } else {
        if (c0 < half) y[c0] = f32_to_bf16_rne(v0);
        if (c1 < half) y[c1] = f32_to_bf16_rne(v1);
      }
    }
}

template <int MT, int KS, bool ACT>
hipError_t launch_rows(const ExpertArgs &g, hipStream_t stream) {
  constexpr int TM = 16 * MT, OUT = (ACT ? 16 : 32) * (8 / KS), PART = 8 * MT * 2 * 1024;
  const int64_t nt = ((ACT ? g.N / 2 : g.N) + OUT - 1) / OUT, mt = g.n / TM + (g.E < g.n ? g.E : g.n);
  if (nt * mt > 0x7fffffff) return hipErrorInvalidConfiguration;
  int ch = 65536 / TM / 1024 * 1024;
  if (ch > (g.K + 1023) / 1024 * 1024) ch = (g.K + 1023) / 1024 * 1024;
  const size_t lds = (size_t)TM * ch > PART || KS == 1 ? (size_t)TM * ch : PART;
  hipLaunchKernelGGL((gemm_experts_rows<MT, KS, ACT>), dim3((unsigned)(nt * mt)), dim3(512), lds, stream, g, ch, (int)nt,
                     div_by((uint32_t)g.per));
  return hipGetLastError();
}

template <bool ACT>
hipError_t launch(const ExpertArgs &g, hipStream_t stream) {
  if (g.n <= 8 * (int64_t)g.E) return launch_rows<1, 2, ACT>(g, stream);
  return launch_rows<4, 1, ACT>(g, stream);
}

}  // namespace

hipError_t launch_gemm_experts(const ExpertArgs &g, int act, hipStream_t stream) {
  return act == OQ_ACT_SWIGLU ? launch<true>(g, stream) : launch<false>(g, stream);
}

}  // namespace oq
