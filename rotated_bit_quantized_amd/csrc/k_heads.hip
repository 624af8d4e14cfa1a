// Per-head norm and rotary embedding, into dense rows or a paged cache
// (oq_qk_norm_rope, oq_kv_append).
//
//   n = x rsqrt(mean(x^2) + eps) w        over the d elements of one head
//   (a, b) -> (a cos - b sin, b cos + a sin)   on the rotary pairs of n
//
// Bound: HBM traffic (2 bytes in and 2 out per element, some ten float32
// operations each).  A head is held by L = 8 .. 64 lanes of one wavefront, 8
// elements (one 16-byte load and store) per lane, so the norm's sum is a few
// cross-lane adds and nothing goes through memory twice.  A lane group takes
// HPG heads of one token: their loads are all issued before the first is
// used, and the token's cos and sin, twice the bytes of a head, are loaded
// once for all of them.
#include "oq_internal.h"

namespace oq {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// How the rotary pairs of a head lie over its lanes.
enum RopeKind : int {
  ROPE_NONE = 0,
  ROPE_SPLIT = 1,  // (i, i + dim/2), dim/2 a multiple of 8: partners are whole lanes
  ROPE_PAIRS = 2,  // (2i, 2i + 1): partners share a lane; dim a multiple of 8
  ROPE_ANY = 3,    // any other even dim: partners are exchanged through LDS
};

// HPG heads of one token per lane group of L lanes.
template <int L, int KIND, int HPG>
__global__ void __launch_bounds__(256) heads_kernel(const HeadArgs a, const int chunks0, const int chunks) {
  __shared__ float stage[KIND == ROPE_ANY ? 256 * 8 : 1];
  const int lane = threadIdx.x & 63;
  const int g = threadIdx.x / L, gl = threadIdx.x % L;  // lane group of the workgroup, lane of the group
  const int64_t item = (int64_t)blockIdx.x * (256 / L) + g;
  const int64_t t = item / chunks;
  if (KIND != ROPE_ANY && t >= a.T) return;
  const bool live = t < a.T;
  const int c = (int)(item - t * chunks);
  const int pi = c >= chunks0 ? 1 : 0;
  const HeadPart &P = a.part[pi];
  const int h0 = (c - (pi ? chunks0 : 0)) * HPG;
  const int nh = P.heads - h0 < HPG ? P.heads - h0 : HPG;
  const int e0 = gl * 8;
  const bool mine = live && e0 < a.d;

  // where the outputs go
  uint16_t *out = nullptr;
  int64_t out_hs = P.out_hs;
  if (live) {
    if (a.slot) {
      const int64_t s = a.slot[t];
      if (s >= 0 && s < a.slots) {
        const int64_t page = s >> a.page_log2, off = s & ((1 << a.page_log2) - 1);
        out_hs = (int64_t)a.d << a.page_log2;
        out = P.out + page * a.page_stride + off * a.d + h0 * out_hs;
      } else if (KIND != ROPE_ANY) {
        return;
      }
    } else {
      out = P.out + t * P.out_ld + h0 * P.out_hs;
    }
  }

  u32x4 raw[HPG];
#pragma unroll
  for (int i = 0; i < HPG; ++i) {
    raw[i] = (u32x4){0u, 0u, 0u, 0u};
    if (mine && i < nh) raw[i] = *reinterpret_cast<const u32x4 *>(P.x + t * P.ld + (h0 + i) * P.hs + e0);
  }

  const bool turn = KIND != ROPE_NONE && P.rope;
  const int dim = a.rope.dim, hd = dim / 2;
  // this lane's cos and sin: element e of a split pair uses index e mod dim/2
  // (8 in a row), element 2i or 2i + 1 of an interleaved one index i (4)
  float co[8], si[8];
  bool bad = false;
  int64_t row = 0;
  if (turn && live) {
    row = a.pos ? a.pos[t] : t;
    bad = row < 0 || row >= a.rope.rows;
    if (bad) row = 0;
  }
  const bool low = e0 < hd;  // split pairs: this lane holds the a side
  if (KIND == ROPE_SPLIT) {
#pragma unroll
    for (int j = 0; j < 8; ++j) co[j] = 1.f, si[j] = 0.f;
    if (turn && mine && e0 < dim) {
      const float *cp = a.rope.cos + row * hd + (low ? e0 : e0 - hd);
      const float *sp = a.rope.sin + row * hd + (low ? e0 : e0 - hd);
#pragma unroll
      for (int j = 0; j < 8; ++j) co[j] = cp[j], si[j] = low ? -sp[j] : sp[j];
    }
  } else if (KIND == ROPE_PAIRS) {
#pragma unroll
    for (int j = 0; j < 4; ++j) co[j] = 1.f, si[j] = 0.f;
    if (turn && mine && e0 < dim) {
      const float *cp = a.rope.cos + row * hd + e0 / 2;
      const float *sp = a.rope.sin + row * hd + e0 / 2;
#pragma unroll
      for (int j = 0; j < 4; ++j) co[j] = cp[j], si[j] = sp[j];
    }
  }

  float w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = (P.w && mine) ? P.w[e0 + j] : 1.f;
  const float inv_d = 1.f / (float)a.d;

#pragma unroll
  for (int i = 0; i < HPG; ++i) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[2 * j] = bf16_lo(raw[i][j]), x[2 * j + 1] = bf16_hi(raw[i][j]);
    if (P.w) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) s = __builtin_fmaf(x[j], x[j], s);
#pragma unroll
      for (int m = 1; m < L; m <<= 1) s += __shfl_xor(s, m);
      const float r = 1.f / __builtin_sqrtf(s * inv_d + a.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
    }
    if (KIND == ROPE_SPLIT) {
      const int src = !turn || e0 >= dim ? lane : low ? lane + hd / 8 : lane - hd / 8;
      float p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = __shfl(x[j], src);
      if (turn) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * co[j] + p[j] * si[j];
      }
    } else if (KIND == ROPE_PAIRS) {
      if (turn) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float u = x[2 * j], v = x[2 * j + 1];
          x[2 * j] = u * co[j] - v * si[j];
          x[2 * j + 1] = v * co[j] + u * si[j];
        }
      }
    } else if (KIND == ROPE_ANY) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) stage[threadIdx.x * 8 + j] = x[j];
      __syncthreads();
      if (turn && mine) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = e0 + j;
          if (e >= dim) continue;
          const bool first = a.rope.interleaved ? !(e & 1) : e < hd;
          const int k = a.rope.interleaved ? e >> 1 : first ? e : e - hd;
          const int pe = a.rope.interleaved ? e ^ 1 : first ? e + hd : e - hd;
          const float cv = a.rope.cos[row * hd + k], sv = a.rope.sin[row * hd + k];
          const float pv = stage[g * L * 8 + pe];
          x[j] = first ? x[j] * cv - pv * sv : x[j] * cv + pv * sv;
        }
      }
    }
    if (turn && bad) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = __builtin_nanf("");
    }
    if (mine && out && i < nh) {
      u32x4 r;
      if (P.w || turn) {
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = (uint32_t)f32_to_bf16_rne(x[2 * j]) | ((uint32_t)f32_to_bf16_rne(x[2 * j + 1]) << 16);
      } else {
        r = raw[i];  // values pass bit for bit
      }
      *reinterpret_cast<u32x4 *>(out + i * out_hs + e0) = r;
    }
  }
}

template <int L, int KIND, int HPG>
hipError_t launch_l(const HeadArgs &a, hipStream_t stream) {
  const int c0 = (a.part[0].heads + HPG - 1) / HPG, c1 = (a.part[1].heads + HPG - 1) / HPG;
  const int64_t items = a.T * (c0 + c1), per = 256 / L;
  const int64_t blocks = (items + per - 1) / per;
  if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((heads_kernel<L, KIND, HPG>), dim3((unsigned)blocks), dim3(256), 0, stream, a, c0, c0 + c1);
  return hipGetLastError();
}

template <int KIND, int HPG>
hipError_t launch_k(const HeadArgs &a, hipStream_t stream) {
  if (a.d <= 64) return launch_l<8, KIND, HPG>(a, stream);
  if (a.d <= 128) return launch_l<16, KIND, HPG>(a, stream);
  if (a.d <= 256) return launch_l<32, KIND, HPG>(a, stream);
  return launch_l<64, KIND, HPG>(a, stream);
}

template <int HPG>
hipError_t launch_h(const HeadArgs &a, int kind, hipStream_t stream) {
  switch (kind) {
    case ROPE_NONE: return launch_k<ROPE_NONE, HPG>(a, stream);
    case ROPE_SPLIT: return launch_k<ROPE_SPLIT, HPG>(a, stream);
    case ROPE_PAIRS: return launch_k<ROPE_PAIRS, HPG>(a, stream);
  }
  return launch_k<ROPE_ANY, HPG>(a, stream);
}

}  // namespace

hipError_t launch_heads(const HeadArgs &a, hipStream_t stream) {
  if (a.T == 0 || a.part[0].heads + a.part[1].heads == 0) return hipSuccess;
  int kind = ROPE_NONE;
  if (a.rope.cos)
    kind = !a.rope.interleaved && a.rope.dim % 16 == 0 ? ROPE_SPLIT
           : a.rope.interleaved && a.rope.dim % 8 == 0 ? ROPE_PAIRS
                                                       : ROPE_ANY;
  return launch_h<1>(a, kind, stream);
}

}  // namespace oq
