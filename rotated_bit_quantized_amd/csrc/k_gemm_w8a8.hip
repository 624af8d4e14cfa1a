// int8 activations x int8 weights on the gfx950 int8 MFMA (oq_gemm_w8a8).
//
//   y[t][o] = bf16( a_scale[t] w_scale[o] acc[t][o] + mean[t] w1[o] + bias[o] )
//   acc = exact int32 sum over K, converted to float32 with one rounding.
#include "oq_internal.h"

namespace oq {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

// One 32 x 32 output tile per wavefront, fragments straight from memory.
__global__ void __launch_bounds__(256)
gemm_w8a8_kernel(const int8_t *__restrict__ qa, int64_t lda, const float *__restrict__ a_scale, int64_t M, int K,
                 const int8_t *__restrict__ w, int64_t ldw, const float *__restrict__ w_scale, int N,
                 const float *__restrict__ mean, const float *__restrict__ w1, const float *__restrict__ bias,
                 uint16_t *__restrict__ y, int64_t ldy) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m0 = (int64_t)blockIdx.y * 64 + 32 * (wave >> 1);
  const int64_t n0 = (int64_t)blockIdx.x * 64 + 32 * (wave & 1);
  const int r = lane & 31, half = lane >> 5;
  const int64_t ar = m0 + r < M ? m0 + r : M - 1, br = n0 + r < N ? n0 + r : N - 1;
  v16i acc = (v16i){};
  for (int k = 0; k < K; k += 32) {
    // the last step of a K that is 16 more than a multiple of 32 has no upper half
    v4i A = (v4i){}, B = (v4i){};
    if (k + 16 * half < K) {
      A = *reinterpret_cast<const v4i *>(qa + ar * lda + k + 16 * half);
      B = *reinterpret_cast<const v4i *>(w + br * ldw + k + 16 * half);
    }
    acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(A, B, acc, 0, 0, 0);
  }
  const int64_t col = n0 + r;
  if (col >= N) return;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int64_t row = m0 + (e >> 2) * 8 + half * 4 + (e & 3);
    if (row >= M) continue;
    float v = a_scale[row] * w_scale[col] * (float)acc[e];
    if (mean) v = __builtin_fmaf(mean[row], w1[col], v);
    if (bias) v = v + bias[col];
    y[row * ldy + col] = f32_to_bf16_rne(v);
  }
}

}  // namespace

hipError_t launch_gemm_w8a8(const int8_t *qa, int64_t lda, const float *a_scale, int64_t M, int K, const int8_t *w,
                            int64_t ldw, const float *w_scale, int N, const float *mean, const float *w1,
                            const float *bias, uint16_t *y, int64_t ldy, hipStream_t stream) {
  dim3 grid((unsigned)((N + 63) / 64), (unsigned)((M + 63) / 64));
  hipLaunchKernelGGL(gemm_w8a8_kernel, grid, dim3(256), 0, stream, qa, lda, a_scale, M, K, w, ldw, w_scale, N, mean, w1,
                     bias, y, ldy);
  return hipGetLastError();
}

}  // namespace oq
