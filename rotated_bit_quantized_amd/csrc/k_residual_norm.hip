// The residual stream between two blocks (oq_residual_norm).
//
//   u = sum_j weights[t][j] y[t k + j]
//   R = r_scale r + y_scale gate post(u),   h = pre(R) (1 + scale) + shift
//
// Bound: HBM traffic, k + 3 bfloat16 rows a token.  L threads hold a row, NV
// pieces of 8 elements each (16-byte loads and stores), so that everything
// between the loads and the stores happens in registers: the sums over the
// row are cross-lane adds, and meet in LDS where L passes a wavefront.  A layer
// norm takes its squares about the mean, a second sum over the same registers.  One
// piece a thread up to 2048 elements, two above.
// Measured: 32768 x 4096, norms on both sides, 194 to 204 us, 5.3 to 5.5 TB/s (a large
// copy: 5.2; four pieces a thread 199, one 203), 8192 x 8192 105 us (four 108, one 130);
// 4100 x 1920 in float32 with gate and modulation 22 us (two pieces 22, four 26); 64 x 8
// x 2048 5.0 us, two trips to memory and a launch (two pieces 6.4, four 8.7).
#include "sparse_plan.h"

namespace oq {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}

// The sum over each group of L threads, in every one of them.  slot: LDS [16],
// another one for each call of a row (a wavefront may still read the last one).
template <int L>
__device__ __forceinline__ float group_sum(float v, float *slot) {
  v = dpp_add<0xB1>(v);                // lane ^ 1
  v = dpp_add<0x4E>(v);                // lane ^ 2
  v = dpp_add<0x141>(v);               // the other quad of 8 (half mirror)
  if (L >= 16) v = dpp_add<0x140>(v);  // the other 8 of 16 (mirror)
  if (L >= 32) v += __shfl_xor(v, 16);
  if (L >= 64) v += __shfl_xor(v, 32);
  if (L > 64) {
    constexpr int W = L > 64 ? L / 64 : 1;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) slot[wave] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += slot[wave / W * W + w];
  }
  return v;
}

__device__ __forceinline__ void unpack8(float (&x)[8], const u32x4 raw) {
#pragma unroll
  for (int j = 0; j < 4; ++j) x[2 * j] = bf16_lo(raw[j]), x[2 * j + 1] = bf16_hi(raw[j]);
}
__device__ __forceinline__ u32x4 pack8(const float (&x)[8]) {
  u32x4 raw;
#pragma unroll
  for (int j = 0; j < 4; ++j) raw[j] = (uint32_t)f32_to_bf16_rne(x[2 * j]) | (uint32_t)f32_to_bf16_rne(x[2 * j + 1]) << 16;
  return raw;
}
__device__ __forceinline__ void load8(float (&x)[8], const float *p) {  // 4-byte aligned
  const f32x4 a = *reinterpret_cast<const f32x4_a4 *>(p), b = *reinterpret_cast<const f32x4_a4 *>(p + 4);
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = a[j], x[4 + j] = b[j];
}

// x through the norm, elements e[v] .. e[v] + 7 of a row (live: inside it)
template <int L, int NV>
__device__ __forceinline__ void norm(float (&x)[NV][8], const oq_norm &n, const int (&e)[NV], int d, float *slots) {
  const float inv_d = 1.f / (float)d;
  if (n.kind == OQ_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += x[v][j];  // zeros outside the row
    const float mean = group_sum<L>(s, slots) * inv_d;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) x[v][j] = e[v] < d ? x[v][j] - mean : 0.f;
  }
  float q = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) q = __builtin_fmaf(x[v][j], x[v][j], q);
  const float inv = 1.f / sqrtf(group_sum<L>(q, slots + 16) * inv_d + n.eps);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    float w[8], b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.f, b[j] = 0.f;
    if (e[v] < d) {
      if (n.w) load8(w, n.w + e[v]);
      if (n.b) load8(b, n.b + e[v]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) x[v][j] = __builtin_fmaf(x[v][j] * inv, w[j], b[j]);
  }
}

template <int L, int NV, bool RBF>
__global__ void __launch_bounds__(L > 256 ? L : 256) residual_norm_kernel(const NormArgs a, const int64_t t0) {
  constexpr int ROWS = L > 256 ? 1 : 256 / L;
  __shared__ float slots[L > 64 ? 4 * 16 : 1];
  const int gl = threadIdx.x % L;
  const int64_t t = t0 + (int64_t)blockIdx.x * ROWS + threadIdx.x / L;
  if (L <= 64 && t >= a.T) return;
  const bool row_live = t < a.T;
  const int d = a.d;
  int e[NV];
  bool live[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) e[v] = 8 * (gl + L * v), live[v] = row_live && e[v] < d;

  // all loads before the first use
  u32x4 raw_y[NV], raw_r[NV][RBF ? 1 : 2];
  const bool one = a.y && !a.weights;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    raw_y[v] = (u32x4){0, 0, 0, 0};
    if (one && live[v]) raw_y[v] = *reinterpret_cast<const u32x4 *>(a.y + t * a.y_ld + e[v]);
    raw_r[v][0] = (u32x4){0, 0, 0, 0};
    if (!RBF) raw_r[v][RBF ? 0 : 1] = (u32x4){0, 0, 0, 0};
    if (a.r && live[v]) {
      if (RBF) {
        raw_r[v][0] = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.r) + t * a.r_ld + e[v]);
      } else {
        const float *p = static_cast<const float *>(a.r) + t * a.r_ld + e[v];
        raw_r[v][0] = *reinterpret_cast<const u32x4 *>(p);
        raw_r[v][RBF ? 0 : 1] = *reinterpret_cast<const u32x4 *>(p + 4);
      }
    }
  }
  int64_t mrow = 0;
  bool bad = false;
  const bool mod = a.mod.gate || a.mod.scale || a.mod.shift;
  if (mod && row_live) {
    mrow = a.mod.row ? a.mod.row[t] : a.mod.rows == 1 ? 0 : t;
    bad = mrow < 0 || mrow >= a.mod.rows;
    if (bad) mrow = 0;
  }

  float x[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) unpack8(x[v], raw_y[v]);
  if (a.y && a.weights) {
    // the rows of an entry without weight are not read; four in flight
    for (int j0 = 0; j0 < a.k; j0 += 4) {
      float w[4];
      u32x4 raw[4][NV];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = row_live && j0 + j < a.k ? a.weights[t * a.k + j0 + j] : 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          raw[j][v] = (u32x4){0, 0, 0, 0};
          if (w[j] != 0.f && live[v]) raw[j][v] = *reinterpret_cast<const u32x4 *>(a.y + (t * a.k + j0 + j) * a.y_ld + e[v]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          float z[8];
          unpack8(z, raw[j][v]);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[v][i] = w[j] != 0.f ? __builtin_fmaf(w[j], z[i], x[v][i]) : x[v][i];
        }
    }
  }
  if (a.post.kind) norm<L, NV>(x, a.post, e, d, slots);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    float r[8], g[8];
    if (RBF) {
      unpack8(r, raw_r[v][0]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = __uint_as_float(raw_r[v][RBF ? 0 : j / 4][j % 4]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = a.y_scale;
    if (a.mod.gate && live[v]) {
      unpack8(g, *reinterpret_cast<const u32x4 *>(a.mod.gate + mrow * a.mod.ld + e[v]));
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] *= a.y_scale;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // without a branch or a residual there is nothing to add: 0 x inf would be NaN
      float z = a.y ? g[j] * x[v][j] : 0.f;
      if (a.r) z = a.y ? __builtin_fmaf(a.r_scale, r[j], z) : a.r_scale * r[j];
      x[v][j] = bad ? NAN : z;
    }
    if (a.r_out && live[v]) {
      if (RBF) {
        *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.r_out) + t * a.ro_ld + e[v]) = pack8(x[v]);
      } else {
        float *p = static_cast<float *>(a.r_out) + t * a.ro_ld + e[v];
        *reinterpret_cast<f32x4 *>(p) = (f32x4){x[v][0], x[v][1], x[v][2], x[v][3]};
        *reinterpret_cast<f32x4 *>(p + 4) = (f32x4){x[v][4], x[v][5], x[v][6], x[v][7]};
      }
    }
    if (!live[v]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[v][j] = 0.f;
    }
  }
  if (!a.h) return;
  if (a.pre.kind) norm<L, NV>(x, a.pre, e, d, slots + (L > 64 ? 32 : 0));
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (!live[v]) continue;
    float s[8], b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = b[j] = 0.f;
    if (a.mod.scale) unpack8(s, *reinterpret_cast<const u32x4 *>(a.mod.scale + mrow * a.mod.ld + e[v]));
    if (a.mod.shift) unpack8(b, *reinterpret_cast<const u32x4 *>(a.mod.shift + mrow * a.mod.ld + e[v]));
#pragma unroll
    for (int j = 0; j < 8; ++j) x[v][j] = __builtin_fmaf(x[v][j], 1.f + s[j], b[j]);
    *reinterpret_cast<u32x4 *>(a.h + t * a.h_ld + e[v]) = pack8(x[v]);
  }
}

template <int L, int NV>
hipError_t launch(const NormArgs &a, bool r_bf16, hipStream_t stream) {
  constexpr int THREADS = L > 256 ? L : 256, ROWS = THREADS / L;
  constexpr int64_t MOST = rows_of_launch(THREADS) * ROWS;
  for (int64_t t0 = 0; t0 < a.T; t0 += MOST) {
    const dim3 grid((unsigned)(((a.T - t0 < MOST ? a.T - t0 : MOST) + ROWS - 1) / ROWS)), block(THREADS);
    if (r_bf16) hipLaunchKernelGGL((residual_norm_kernel<L, NV, true>), grid, block, 0, stream, a, t0);
    else hipLaunchKernelGGL((residual_norm_kernel<L, NV, false>), grid, block, 0, stream, a, t0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_residual_norm(const NormArgs &a, bool r_bf16, hipStream_t stream) {
  const int pieces = a.d / 8;
  if (pieces <= 8) return launch<8, 1>(a, r_bf16, stream);
  if (pieces <= 16) return launch<16, 1>(a, r_bf16, stream);
  if (pieces <= 32) return launch<32, 1>(a, r_bf16, stream);
  if (pieces <= 64) return launch<64, 1>(a, r_bf16, stream);
  if (pieces <= 128) return launch<128, 1>(a, r_bf16, stream);
  if (pieces <= 256) return launch<256, 1>(a, r_bf16, stream);
  if (pieces <= 512) return launch<256, 2>(a, r_bf16, stream);
  if (pieces <= 1024) return launch<512, 2>(a, r_bf16, stream);
  return launch<1024, 2>(a, r_bf16, stream);
}

}  // namespace oq
