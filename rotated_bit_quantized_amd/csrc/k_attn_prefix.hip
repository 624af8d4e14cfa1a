// Attention of a batch that shares a prefix of a paged cache (oq_attn_prefix).
#include "oq_internal.h"

namespace oq {
namespace {

// One query row per wavefront, one key per step, the head over the lanes.
template <int D>
__global__ void __launch_bounds__(256) attn_row_kernel(const AttnArgs a) {
  constexpr int E = D / 64;
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t T = (int64_t)a.B * a.n_q;
  if (row >= T * a.heads_q) return;
  const int64_t t = row / a.heads_q;
  const int h = (int)(row - t * a.heads_q), b = (int)(t / a.n_q), i = (int)(t - (int64_t)b * a.n_q);
  const int hk = h / (a.heads_q / a.kv.heads);
  float q[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = bf16_lo(a.q[t * a.q_ld + h * a.q_hs + lane + 64 * e]);
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int part = 0; part < 2; ++part) {
    const int32_t *table = part ? a.tables + (int64_t)b * a.table_ld : a.prefix_table;
    int64_t n = a.prefix_len;
    if (part) {
      n = a.table_ld ? (int64_t)a.lens[b] - a.n_q + 1 + i : 0;
      if (n > (int64_t)a.table_ld * a.kv.page) n = (int64_t)a.table_ld * a.kv.page;
    }
    for (int64_t j = 0; j < n; ++j) {
      const int page = table[j / a.kv.page];
      if ((unsigned)page >= (unsigned)a.kv.pages) continue;
      const int64_t at = page * a.kv.page_stride + ((int64_t)hk * a.kv.page + j % a.kv.page) * D + lane;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = __builtin_fmaf(q[e], bf16_lo(a.kv.k[at + 64 * e]), s);
#pragma unroll
      for (int x = 1; x < 64; x <<= 1) s += __shfl_xor(s, x);
      s *= a.scale;
      const float mn = fmaxf(m, s);
      if (mn == -INFINITY) continue;
      const float c = expf(m - mn), p = expf(s - mn);
      m = mn;
      l = l * c + p;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = acc[e] * c + p * bf16_lo(a.kv.v[at + 64 * e]);
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    a.o[t * a.o_ld + h * a.o_hs + lane + 64 * e] = f32_to_bf16_rne(m == -INFINITY ? 0.f : acc[e] / l);
  if (a.lse && lane == 0) a.lse[row] = m == -INFINITY ? -INFINITY : m + logf(l);
}

}  // namespace

size_t attn_prefix_ws(const AttnArgs &) { return 0; }

hipError_t launch_attn_prefix(const AttnArgs &a, void *, hipStream_t stream) {
  const int64_t rows = (int64_t)a.B * a.n_q * a.heads_q;
  const dim3 grid((unsigned)((rows + 3) / 4));
  if (a.kv.d == 64) hipLaunchKernelGGL(attn_row_kernel<64>, grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL(attn_row_kernel<128>, grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace oq
