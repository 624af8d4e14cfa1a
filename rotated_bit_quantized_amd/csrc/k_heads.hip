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
// used, and the token's cos and sin, four times the bytes of a head, are
// loaded once for all of them.  A workgroup is 256 / L tokens of the same
// heads, so which tensor and which heads is scalar.
// Measured: 32768 tokens of 32 + 8 heads of 128 145 us, 4.8 TB/s (a large copy:
// 5.2); into the cache, 8 + 8 heads, 66 us, 4.3 TB/s.
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

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}

// the sum over each group of L lanes, in every lane of it
template <int L>
__device__ __forceinline__ float group_sum(float v) {
  v = dpp_add<0xB1>(v);                 // lane ^ 1
  v = dpp_add<0x4E>(v);                 // lane ^ 2
  v = dpp_add<0x141>(v);                // the other quad of 8 (half mirror)
  if (L >= 16) v = dpp_add<0x140>(v);   // the other 8 of 16 (mirror)
  if (L >= 32) v += __shfl_xor(v, 16);
  if (L >= 64) v += __shfl_xor(v, 32);
  return v;
}

__device__ __forceinline__ void load_f32(float *dst, const float *src, int n) {
#pragma unroll
  for (int j = 0; j < n; ++j) dst[j] = src[j];
}

__device__ __forceinline__ void unpack8(float (&x)[8], const u32x4 raw) {
#pragma unroll
  for (int j = 0; j < 4; ++j) x[2 * j] = bf16_lo(raw[j]), x[2 * j + 1] = bf16_hi(raw[j]);
}

// HPG heads of one token per lane group of L lanes.
template <int L, int KIND, int HPG>
__global__ void __launch_bounds__(256) heads_kernel(const HeadArgs a, const int64_t t0, const int chunks0, const int chunks) {
  __shared__ float stage[KIND == ROPE_ANY ? 256 * 8 : 1];
  const int lane = threadIdx.x & 63;
  const int g = threadIdx.x / L, gl = threadIdx.x % L;  // lane group of the workgroup, lane of the group
  const int c = blockIdx.x % chunks;
  const int64_t t = t0 + (int64_t)(blockIdx.x / chunks) * (256 / L) + g;
  if (KIND != ROPE_ANY && t >= a.T) return;
  const bool live = t < a.T;
  const int pi = c >= chunks0 ? 1 : 0;
  const HeadPart &P = a.part[pi];
  const int h0 = (c - (pi ? chunks0 : 0)) * HPG;
  const int nh = P.heads - h0 < HPG ? P.heads - h0 : HPG;
  const int e0 = gl * 8;
  const bool mine = live && e0 < a.d;

  u32x4 raw[HPG];
  const uint16_t *src = P.x + t * P.ld + h0 * P.hs + e0;
#pragma unroll
  for (int i = 0; i < HPG; ++i) {
    raw[i] = (u32x4){0u, 0u, 0u, 0u};
    if (mine && i < nh) raw[i] = *reinterpret_cast<const u32x4 *>(src + i * P.hs);
  }

  // where the outputs go
  uint16_t *out = nullptr;
  int64_t out_hs = P.out_hs;
  if (live) {
    if (a.slot) {
      const int64_t s = a.slot[t];
      out_hs = (int64_t)a.d << a.page_log2;
      if (s >= 0 && s < a.slots) {
        const int64_t page = s >> a.page_log2, off = s & ((1 << a.page_log2) - 1);
        out = P.out + page * a.page_stride + off * a.d + h0 * out_hs + e0;
      }
    } else {
      out = P.out + t * P.out_ld + h0 * P.out_hs + e0;
    }
  }

  const bool turn = KIND != ROPE_NONE && P.rope;
  const int dim = a.rope.dim, hd = dim / 2;
  bool bad = false;
  int64_t row = 0;
  if (turn && live) {
    row = a.pos ? a.pos[t] : t;
    bad = row < 0 || row >= a.rope.rows;
    if (bad) row = 0;
  }
  // this lane's cos and sin: element e of a split pair uses index e mod dim/2
  // (8 in a row, sin negated on the a side), element 2i or 2i + 1 of an
  // interleaved one index i (4 in a row); otherwise element by element
  constexpr int CN = KIND == ROPE_PAIRS ? 4 : 8;
  float co[CN], si[CN];
  const bool low = e0 < hd, rot = turn && mine && e0 < dim;  // others pass: turning an infinity by 0 would make NaN
  int partner = lane;  // the lane that holds the other side of this lane's split pairs
  if (KIND == ROPE_SPLIT || KIND == ROPE_PAIRS) {
#pragma unroll
    for (int j = 0; j < CN; ++j) co[j] = 1.f, si[j] = 0.f;
    if (rot) {
      const int at = KIND == ROPE_PAIRS ? e0 / 2 : low ? e0 : e0 - hd;
      load_f32(co, a.rope.cos + row * hd + at, CN);
      load_f32(si, a.rope.sin + row * hd + at, CN);
      if (KIND == ROPE_SPLIT) {
        partner = low ? lane + hd / 8 : lane - hd / 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) si[j] = low ? -si[j] : si[j];
      }
    }
  }
  if (KIND == ROPE_ANY) {
#pragma unroll
    for (int j = 0; j < CN; ++j) {
      const int e = e0 + j;
      co[j] = 1.f, si[j] = 0.f;
      if (!rot || e >= dim) continue;
      const bool first = a.rope.interleaved ? !(e & 1) : e < hd;
      const int64_t k = row * hd + (a.rope.interleaved ? e >> 1 : first ? e : e - hd);
      co[j] = a.rope.cos[k];
      si[j] = first ? -a.rope.sin[k] : a.rope.sin[k];
    }
  }

  float w[8], wp[KIND == ROPE_SPLIT ? 8 : 1];  // the norm weights of this lane's elements and of its partner's
  if (P.w && mine) {
    load_f32(w, P.w + e0, 8);
    if (KIND == ROPE_SPLIT) load_f32(wp, P.w + e0 + 8 * (partner - lane), 8);
  }
  const float inv_d = 1.f / (float)a.d;

#pragma unroll
  for (int i = 0; i < HPG; ++i) {
    float x[8];
    unpack8(x, raw[i]);
    float r = 1.f;
    if (P.w) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) s = __builtin_fmaf(x[j], x[j], s);
      r = 1.f / __builtin_sqrtf(group_sum<L>(s) * inv_d + a.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
    }
    if (KIND == ROPE_SPLIT && turn) {
      u32x4 pr;
#pragma unroll
      for (int j = 0; j < 4; ++j) pr[j] = __shfl(raw[i][j], partner);
      float p[8];
      unpack8(p, pr);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float y = x[j] * co[j] + (P.w ? p[j] * r * wp[j] : p[j]) * si[j];
        x[j] = rot ? y : x[j];
      }
    } else if (KIND == ROPE_PAIRS && turn) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float u = x[2 * j], v = x[2 * j + 1], y = u * co[j] - v * si[j], z = v * co[j] + u * si[j];
        x[2 * j] = rot ? y : u;
        x[2 * j + 1] = rot ? z : v;
      }
    } else if (KIND == ROPE_ANY && P.rope) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) stage[threadIdx.x * 8 + j] = x[j];
      __syncthreads();
      if (mine) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = e0 + j;
          if (e >= dim) continue;
          const int pe = a.rope.interleaved ? e ^ 1 : e < hd ? e + hd : e - hd;
          x[j] = x[j] * co[j] + stage[g * L * 8 + pe] * si[j];
        }
      }
    }
    if (mine && out && i < nh) {
      u32x4 y;
      if (P.w || turn) {
        if (bad) {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = __builtin_nanf("");
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = (uint32_t)f32_to_bf16_rne(x[2 * j]) | ((uint32_t)f32_to_bf16_rne(x[2 * j + 1]) << 16);
      } else {
        y = raw[i];  // values pass bit for bit
      }
      // streamed: 4 to 8% faster than cached stores on 32768 tokens, no slower on 64
      __builtin_nontemporal_store(y, reinterpret_cast<u32x4 *>(out + i * out_hs));
    }
  }
}

template <int L, int KIND, int HPG>
hipError_t launch_l(const HeadArgs &a, hipStream_t stream) {
  const int c0 = (a.part[0].heads + HPG - 1) / HPG, c1 = (a.part[1].heads + HPG - 1) / HPG;
  const int64_t per = 256 / L, most = rows_of_launch(256 * (c0 + c1)) * per;  // tokens of a launch
  for (int64_t t0 = 0; t0 < a.T; t0 += most) {
    const int64_t blocks = ((a.T - t0 < most ? a.T - t0 : most) + per - 1) / per * (c0 + c1);
    hipLaunchKernelGGL((heads_kernel<L, KIND, HPG>), dim3((unsigned)blocks), dim3(256), 0, stream, a, t0, c0, c0 + c1);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
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
  const int64_t heads = a.part[0].heads + a.part[1].heads;
  if (a.T == 0 || heads == 0) return hipSuccess;
  int kind = ROPE_NONE;
  if (a.rope.cos)
    kind = !a.rope.interleaved && a.rope.dim % 16 == 0 ? ROPE_SPLIT
           : a.rope.interleaved && a.rope.dim % 8 == 0 ? ROPE_PAIRS
                                                       : ROPE_ANY;
  // Heads per lane group, by the wavefronts that one head each would take: more
  // heads keep more loads in flight and read the tables less often, fewer give
  // small calls enough wavefronts.  40 heads of 128, one / two / four per group:
  // T = 128 3.3 / 3.5 / 4.9 us, 1024 6.0 / 5.5 / 6.3, 4096 21.7 / 20.1 / 18.6.
  // No more than a part has: 29681 tokens of 1 + 1 heads 12.2 us, 14.3 with two.
  const int64_t waves = a.T * heads * (a.d <= 64 ? 8 : a.d <= 128 ? 16 : a.d <= 256 ? 32 : 64) / 64;
  const int most = a.part[0].heads > a.part[1].heads ? a.part[0].heads : a.part[1].heads;
  if (waves >= 16384 && most > 2) return launch_h<4>(a, kind, stream);
  if (waves >= 4096 && most > 1) return launch_h<2>(a, kind, stream);
  return launch_h<1>(a, kind, stream);
}

}  // namespace oq
