// Log probabilities, ranks, entropy and best alternatives of rows of logits
// (oq_logprobs).
//
//   z = scale log2(e) (x - M),  r = sum 2^z - 1,  t = sum 2^z z     (M: the largest)
//   lse = scale M + log1p(r),  log p = scale (x - M) - log1p(r),  entropy = log1p(r) - ln2 t / (1 + r)
//
// The 1 of r is the largest logit's own term, which is left out of the sum: of a
// nearly certain token all digits of log p are those of r.  Both parts of log p are
// <= 0 and both of the entropy >= 0, so nothing cancels and no sign is ever wrong.
//
// Bound: HBM, one pass over the logits; some 11 vector instructions an element
// (the exponential counts four) are near that.  A workgroup takes a part of a row, its
// pieces of 16 bytes all in flight at once and held in registers as they came: the
// maximum is known before the first exponential, so nothing is rescaled, and what comes
// after it (ranks, best alternatives) reads registers.  Measured: 2048 x 131072
// bfloat16 119 to 135 us by cards and by what ran before, 7 of them the join (4.0 to 4.5
// TB/s; with values unpacked once and kept, one workgroup a CU, 550); 77 x 100003 12 and
// 5; 1 x 32000 float32 8, a launch.  Comparisons below and at the plan are of ten calls in
// a graph on one card, where the first takes 127 to 130.
//
// Alternatives: the `top`-th largest of 64 maxima (over the threads of one lane
// number) is a threshold that at least `top` elements reach and hardly more do.  The
// threads that hold one put their pieces into LDS, where all look through them; what
// reaches the threshold is ranked as whole numbers (value, then falling index), so
// ties never depend on the time.  Rows in which more than the list holds reach the
// threshold (many equal values, or the best ones all in one lane's places) get the
// exact value by bisection, and of values equal to it the first ones in order.
//
// Rows of several parts leave statistics and sorted candidates for a second
// launch, a wavefront a row.
#include "sparse_plan.h"

namespace oq {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float LN2 = 0.693147180559945309417f;

// What is known of a row or a part of it.
struct Part {
  float top;      // the largest logit; 0 where there is nothing but -inf
  float rest, t;  // r and t of above; r is -1 where there is nothing but -inf
  float unused;
};
constexpr float NOTHING = -1.f;  // as rest

// The reference of logits of which `top` is the largest; of nothing but -inf any does.
__device__ __forceinline__ float about(float top) { return top == -INFINITY ? 0.f : top; }

struct Scratch {
  Part *part;      // [T][parts]
  uint64_t *keys;  // [T][parts][top], falling; 0: none
  int32_t *ranks;  // [T][parts][n]
};

// Order-preserving whole numbers, -0 as 0; NaN below all numbers (1).
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return v != v ? 1u : (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) { return k <= 1 ? NAN : __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k); }
__device__ __forceinline__ uint64_t key_of(float v, int i) { return (uint64_t)order_of(v) << 32 | (uint32_t)~i; }

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
  return v > o ? v : o;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = dpp_max<0xB1, 0xF>(v);   // lane ^ 1
  v = dpp_max<0x4E, 0xF>(v);   // lane ^ 2
  v = dpp_max<0x141, 0xF>(v);  // half mirror of 8
  v = dpp_max<0x140, 0xF>(v);  // mirror of 16
  v = dpp_max<0x142, 0xA>(v);  // last lane of the row before, to rows 1 and 3
  v = dpp_max<0x143, 0xC>(v);  // lane 31 to rows 2 and 3
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
template <class T>
__device__ __forceinline__ float logit(const T *row, int i) {
  if constexpr (sizeof(T) == 2) return __uint_as_float((uint32_t)row[i] << 16);
  else return row[i];
}

// log(1 + r) for r >= 0 within 2.7 units of 2^-24 of itself, and -inf of NOTHING: the
// logarithm of the rounded sum and what the rounding left out of it, or three terms of
// the series (log1pf takes 2048 x 131072 another 9 us).
__device__ __forceinline__ float log_sum(float r) {
  const float u = 1.f + r;
  const float far = __builtin_fmaf(__builtin_amdgcn_logf(u), LN2, (r - (u - 1.f)) * __builtin_amdgcn_rcpf(u));
  const float near = r * __builtin_fmaf(r, __builtin_fmaf(r, 1.f / 3.f, -0.5f), 1.f);
  return r == NOTHING ? -INFINITY : r < 0x1p-8f ? near : far;
}
// What a row's statistics, log_s = log_sum(rest) among them, say of a logit and of the row.
__device__ __forceinline__ float log_prob(float x, float scale, const Part &r, float log_s) {
  const float d = x - r.top;
  // a distance past float32 may have a product that is not (if scale < 1; else both are -inf)
  const float z = fabsf(d) < INFINITY || !(fabsf(x) < INFINITY) ? d * scale : __builtin_fmaf(x, scale, -(r.top * scale));
  return z - log_s;
}
__device__ __forceinline__ void row_outputs(const LogprobArgs &a, int64_t t, const Part &r, float log_s) {
  if (a.lse) a.lse[t] = __builtin_fmaf(r.top, a.scale, log_s);
  if (a.entropy) a.entropy[t] = log_s - r.t / (1.f + r.rest) * LN2;
}
template <class T>
__device__ __forceinline__ void token_outputs(const LogprobArgs &a, const T *row, int64_t t, int i, const Part &r, float log_s, int rank) {
  const int tok = a.tokens[t * a.n + i];
  const bool in = tok >= 0 && tok < a.V;
  a.logprob[t * a.n + i] = in ? log_prob(logit(row, tok), a.scale, r, log_s) : NAN;
  a.rank[t * a.n + i] = in ? rank : -1;
}

// The largest of two float32 or four times two bfloat16 numbers at a time; the
// latter as whole numbers: signed ones order all but negative bfloat16 among
// themselves, of which the smallest unsigned one is the largest.
typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

template <class T, int NV>
__device__ __forceinline__ float largest(const u32x4 (&raw)[NV]) {
  float m = -INFINITY;
  if constexpr (sizeof(T) == 2) {
    s16x2 hi = {-32768, -32768};
    u16x2 lo = {65535, 65535};
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w = raw[v][j];
        hi = __builtin_elementwise_max(hi, __builtin_bit_cast(s16x2, w));
        lo = __builtin_elementwise_min(lo, __builtin_bit_cast(u16x2, w));
      }
    const int h = hi.x > hi.y ? hi.x : hi.y;
    const uint32_t l = lo.x < lo.y ? lo.x : lo.y;
    m = __uint_as_float((h < 0 ? l : (uint32_t)h) << 16);
    if (m == m) return m;
    m = -INFINITY;  // a NaN is there: it is passed over
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 4; ++j) m = fmaxf(m, fmaxf(bf16_lo(raw[v][j]), bf16_hi(raw[v][j])));
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 4; ++j) m = fmaxf(m, __uint_as_float(raw[v][j]));  // passes NaN over
  }
  return m;
}

// Pieces part * each .. (part + 1) * each - 1 of a row (from row t0 on), NV a thread at most, by
// WAVES wavefronts.  24 wavefronts fit a CU, three workgroups of 8 or six of 4, whose loads
// run under each other's arithmetic (2048 x 131072 with 32 wavefronts, whose 64
// registers a thread spill: a fifth more).
template <class T, int NV, int WAVES>
__global__ void __launch_bounds__(64 * WAVES, WAVES <= 8 ? 6 : 4) logprobs_part(const LogprobArgs a, const Scratch ws, const int64_t t0, const int parts, const int each) {
  constexpr int THREADS = 64 * WAVES, LIST = THREADS < 512 ? THREADS : 512;  // a thread for each listed candidate
  constexpr int VE = 16 / sizeof(T);  // elements of a piece
  constexpr int HELD = 64;            // threads whose pieces go to LDS for their candidates
  __shared__ u32x4 s_held[HELD * NV];
  __shared__ int s_first[HELD];
  __shared__ uint32_t s_max[WAVES * 64];
  __shared__ float s_sum[3 * WAVES];
  __shared__ uint64_t s_list[LIST];
  __shared__ int s_rank[64];
  __shared__ int s_count[3];  // listed candidates, a count, threads held
  __shared__ uint32_t s_limit;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t in_launch = blockIdx.x / parts;
  const int64_t t = t0 + in_launch;
  const int part = blockIdx.x - in_launch * parts;
  const T *row = static_cast<const T *>(a.logits) + t * a.ld;
  // pieces lie on 16-byte boundaries: the first one may begin before the row
  const int lead = (int)(reinterpret_cast<uintptr_t>(row) & 15) / (int)sizeof(T);
  const int begin = part * each * VE - lead > 0 ? part * each * VE - lead : 0;  // elements of the part
  const int end = (part + 1) * each * VE - lead < a.V ? (part + 1) * each * VE - lead : a.V;
  const int p0 = part * each + (int)threadIdx.x;  // this thread's pieces: p0, p0 + THREADS, ..
  constexpr uint32_t NONE = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;  // -inf
  const u32x4 *pieces = reinterpret_cast<const u32x4 *>(row - lead) + p0;
  const int whole = (end + lead) / VE;                                   // the part's pieces up to here are whole
  const int nv = whole > p0 ? (whole - p0 + THREADS - 1) / THREADS : 0;  // and so many of this thread
  const bool cut = p0 == 0 && lead > 0;                                  // the row begins inside the first one
  u32x4 raw[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    raw[v] = (u32x4){NONE, NONE, NONE, NONE};
    if (v < nv && !(v == 0 && cut)) raw[v] = pieces[v * THREADS];
  }
  // a row's first and last piece, which it may fill in part
  auto partial = [&](int i) {
    u32x4 piece = {NONE, NONE, NONE, NONE};
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      if (i + j < 0 || i + j >= end) continue;
      if constexpr (sizeof(T) == 2) {
        const uint32_t w = piece[j / 2], e = row[i + j];
        piece[j / 2] = j & 1 ? (w & 0xFFFFu) | e << 16 : (w & 0xFFFF0000u) | e;
      } else {
        piece[j] = __float_as_uint(row[i + j]);
      }
    }
    return piece;
  };
  if (cut) raw[0] = partial(-lead);
  if (whole * VE - lead < end && whole >= p0 && (whole - p0) % THREADS == 0 && !(whole == 0 && cut)) {
    const u32x4 piece = partial(whole * VE - lead);
#pragma unroll
    for (int v = 0; v < NV; ++v) raw[v] = v == nv ? piece : raw[v];
  }
  auto at = [&](int v, int j) {
    if constexpr (sizeof(T) == 2) return j & 1 ? bf16_hi(raw[v][j / 2]) : bf16_lo(raw[v][j / 2]);
    else return __uint_as_float(raw[v][j]);
  };
  // what was unpacked of a piece for one pass over the registers is not kept for the next
  auto forget = [&](int v) { asm volatile("" : "+v"(raw[v])); };
  if (threadIdx.x < 64) s_rank[threadIdx.x] = 0;
  if (threadIdx.x < 3) s_count[threadIdx.x] = 0;

  const float mine = largest<T, NV>(raw);
  s_max[threadIdx.x] = order_of(mine);
  __syncthreads();
  uint32_t group = 0;  // the largest over the threads of this lane number
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    const uint32_t o = s_max[64 * w + lane];
    group = o > group ? o : group;
  }
  const float top = value_of(wave_max(group)), ref = about(top), c = a.scale * ATTN_LOG2E;

  // the threshold: the top-th largest of the 64 group maxima
  if (a.top > 0 && wave == 0) {
    uint32_t left = group, limit = 0;
    for (int j = 0; j < a.top; ++j) {
      limit = wave_max(left);
      const int win = __ffsll((long long)__ballot(left == limit)) - 1;
      if (lane == win) left = 0;
    }
    if (lane == 0) s_limit = limit;
  }

  // s and t over all but the largest ones, which are counted.  z is taken about m =
  // RN(ref c) in one step, whose only rounding is z's, and m's error off the sums
  // afterwards: up to |m| = 2^20, where it is below 2^-4.  The elements of a thread that
  // holds a largest one are then summed again, a lane each; of many such threads, and
  // beyond 2^20, every element is looked at (2048 x 131072: 128 us; 140 where every
  // wavefront with a largest one looks at all of its elements).
  float s = 0.f, sum_t = 0.f;
  int largest_ones = 0;
  auto sums = [&](auto add) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      forget(v);
#pragma unroll
      for (int j = 0; j < VE; ++j) add(at(v, j));
    }
  };
  auto add = [&](float z) {
    const float e = __builtin_amdgcn_exp2f(z);
    s += e;
    sum_t = __builtin_fmaf(e, fmaxf(z, -1024.f), sum_t);  // 2^-inf takes no part
  };
  const float m = ref * c;
  const uint64_t owners = __ballot(mine == ref);
  if (fabsf(m) < 0x1p20f && __popcll(owners) <= HELD / WAVES) {
    u32x4 *own = s_held + wave * (HELD / WAVES * NV);  // nobody else's until the next barrier
    if (mine == ref) {
      u32x4 *to = own + NV * __popcll(owners & ((1ull << lane) - 1));
#pragma unroll
      for (int v = 0; v < NV; ++v) to[v] = raw[v];
    }
    sums([&](float x) { add(__builtin_fmaf(x, c, -m)); });
    if (mine == ref) s = sum_t = 0.f;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    for (int h = 0; h < __popcll(owners); ++h) {
      const float x = lane < NV * VE ? logit(reinterpret_cast<const T *>(own + h * NV), lane) : -INFINITY;
      add(x == ref ? -INFINITY : __builtin_fmaf(x, c, -m));
      largest_ones += __popcll(__ballot(x == ref));
    }
    const float off = __builtin_fmaf(ref, c, -m), back = __builtin_amdgcn_exp2f(-off);
    sum_t = back * __builtin_fmaf(-off, s, sum_t);
    s *= back;
  } else {
    sums([&](float x) {
      add(x == ref ? -INFINITY : (x - ref) * c);
      largest_ones += __popcll(__ballot(x == ref));
    });
  }
  s = wave_sum(s);
  sum_t = wave_sum(sum_t);
  if (lane == 0) s_sum[wave] = s, s_sum[WAVES + wave] = sum_t, s_sum[2 * WAVES + wave] = (float)largest_ones;

  // ranks: elements above the token's, and equal ones before it.  A piece before
  // the token's counts from its value on, that one and those behind it from the
  // next value on.  A wavefront whose largest is below the token has nothing to count.
#pragma unroll 1
  for (int i = 0; i < a.n; ++i) {
    const int tok = a.tokens[t * a.n + i];
    if (tok < 0 || tok >= a.V) continue;
    const float xt = logit(row, tok);
    int count = 0;
    if (xt > -INFINITY) {
      const int own = (tok + lead) / VE;  // the token's piece; equal ones in it:
      if (own >= part * each && own < (part + 1) * each && (int)threadIdx.x < VE) {
        const int e = own * VE - lead + (int)threadIdx.x;
        if (e >= 0 && e < tok && logit(row, e) == xt) atomicAdd(s_rank + i, 1);
      }
      if (__ballot(mine >= xt) == 0) continue;
      const float above = value_of(order_of(xt) + 1);
      const int before = own > p0 ? (own - p0 + THREADS - 1) / THREADS : 0;  // pieces of this thread before it
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        forget(v);
        const float limit = v < before ? xt : above;
#pragma unroll
        for (int j = 0; j < VE; ++j) count += __popcll(__ballot(at(v, j) >= limit));
      }
    } else {  // -inf or NaN: no value in the registers stands for places outside the row
      const uint32_t ot = order_of(xt);
      for (int e = begin + (int)threadIdx.x; e < end; e += THREADS) {
        const uint32_t o = order_of(logit(row, e));
        count += o > ot || (o == ot && e < tok);
      }
      for (int o = 32; o; o >>= 1) count += __shfl_xor(count, o);
    }
    if (lane == 0 && count) atomicAdd(s_rank + i, count);
  }
  __syncthreads();
  int n_list = 0, rank = 0;  // of the listed candidates, a thread each
  uint64_t key = 0;
  if (a.top > 0) {
    const uint32_t lowest = order_of(-INFINITY);
    uint32_t limit = s_limit;
    auto add = [&](float x, int i) {
      const int n = atomicAdd(s_count, 1);
      if (n < LIST) s_list[n] = key_of(x, i);
    };
    // the threads that hold a candidate hand their pieces to all; of masked rows
    // every number is one
    const float v0 = value_of(limit > lowest ? limit : lowest + 1);
    if (mine >= v0) {
      const int at_held = atomicAdd(s_count + 2, 1);
      if (at_held < HELD) {
        s_first[at_held] = p0 * VE - lead;
#pragma unroll
        for (int v = 0; v < NV; ++v) s_held[at_held * NV + v] = raw[v];
      }
    }
    __syncthreads();
    const int held = s_count[2];
    bool listed = held <= HELD;
    if (listed) {
      for (int e = threadIdx.x; e < held * (NV * VE); e += THREADS) {
        const int h = e / (NV * VE), r = e - h * (NV * VE);
        float x;
        if constexpr (sizeof(T) == 2) x = __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(s_held)[e] << 16);
        else x = reinterpret_cast<const float *>(s_held)[e];
        if (x >= v0) add(x, s_first[h] + r / VE * (THREADS * VE) + r % VE);
      }
      __syncthreads();
      listed = s_count[0] <= LIST;
      __syncthreads();
    }
    // What is left is rare and reads the part again, element by element.
    // the first `want` elements of order o among this wavefront's, by index
    auto collect_first = [&](uint32_t o, int want) {
      for (int i0 = begin + 64 * wave; i0 < end && want > 0; i0 += THREADS) {
        const int i = i0 + lane;
        const bool hit = i < end && order_of(logit(row, i)) == o;
        const uint64_t hits = __ballot(hit);
        if (hit && __popcll(hits & ((1ull << lane) - 1)) < want) add(value_of(o), i);
        want -= __popcll(hits);
      }
    };
    if (!listed) {
      // too many: the exact top-th value, unless fewer are above the limit
      auto count_from = [&](uint32_t from) {  // how many numbers of order `from` on
        const float least = value_of(from);
        int count = 0;
#pragma unroll 8
        for (int i = begin + (int)threadIdx.x; i < end; i += THREADS) count += logit(row, i) >= least;
        for (int o = 32; o; o >>= 1) count += __shfl_xor(count, o);
        __syncthreads();
        if (threadIdx.x == 0) s_count[1] = 0;
        __syncthreads();
        if (lane == 0) atomicAdd(s_count + 1, count);
        __syncthreads();
        return s_count[1];
      };
      int above = count_from(limit + 1);
      if (above >= a.top) {
        uint32_t lo = limit + 1, hi = order_of(top) + 1;  // count(lo) >= top, count(hi) = 0
        while (hi - lo > 1) {
          const uint32_t mid = lo + (hi - lo) / 2;
          if (count_from(mid) >= a.top) lo = mid;
          else hi = mid;
        }
        limit = lo;
        above = count_from(limit + 1);
      }
      __syncthreads();
      if (threadIdx.x == 0) s_count[0] = 0;
      __syncthreads();
      if (above > 0) {
        const float least = value_of(limit + 1);
        for (int i = begin + (int)threadIdx.x; i < end; i += THREADS) {
          const float x = logit(row, i);
          if (x >= least) add(x, i);
        }
      }
      __syncthreads();
    }
    // fewer than wanted: the first ones equal to the limit, then NaN
    int have = s_count[0];
    __syncthreads();
    if (have < a.top) {
      collect_first(limit, a.top - have);
      __syncthreads();
      have = s_count[0];
      __syncthreads();
      if (have < a.top) collect_first(1, a.top - have);
      __syncthreads();
    }
    n_list = s_count[0];
    if (64 * wave < n_list) {
      key = (int)threadIdx.x < n_list ? s_list[threadIdx.x] : 0;
      for (int j = 0; j < n_list; ++j) rank += s_list[j] > key;
    }
    if (parts > 1) {
      uint64_t *keys = ws.keys + ((int64_t)t * parts + part) * a.top;
      if ((int)threadIdx.x < n_list && rank < a.top) keys[rank] = key;
      if ((int)threadIdx.x >= n_list && (int)threadIdx.x < a.top) keys[threadIdx.x] = 0;
    }
  }
  // the first wavefront's threads have the row's or part's values, those of the list alternatives
  if (wave > 0 && (parts > 1 || 64 * wave >= n_list)) return;
  Part stat{ref, 0.f, 0.f, 0.f};
  float ones = 0.f;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) stat.rest += s_sum[w], stat.t += s_sum[WAVES + w], ones += s_sum[2 * WAVES + w];
  stat.rest = top == INFINITY ? NAN : stat.rest + (ones - 1.f);
  const float log_s = log_sum(stat.rest);
  if (parts == 1) {
    if ((int)threadIdx.x < n_list && rank < a.top) {
      a.top_id[t * a.top + rank] = (int32_t)~(uint32_t)key;
      a.top_logprob[t * a.top + rank] = log_prob(value_of((uint32_t)(key >> 32)), a.scale, stat, log_s);
    }
    if (threadIdx.x == 0) row_outputs(a, t, stat, log_s);
    if ((int)threadIdx.x < a.n) token_outputs(a, row, t, threadIdx.x, stat, log_s, s_rank[threadIdx.x]);
  } else {
    if (threadIdx.x == 0) ws.part[t * parts + part] = stat;
    if ((int)threadIdx.x < a.n) ws.ranks[(t * parts + part) * a.n + threadIdx.x] = s_rank[threadIdx.x];
  }
}

// A wavefront joins a row's parts.  Everything it reads is asked for before it is
// used, but a token's logit.
template <class T>
__global__ void __launch_bounds__(64) logprobs_join(const LogprobArgs a, const Scratch ws, const int parts) {
  extern __shared__ uint64_t s_keys[];  // [parts][top]
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  const T *row = static_cast<const T *>(a.logits) + t * a.ld;
  const int total = parts * a.top;
  const int tok = lane < a.n ? a.tokens[t * a.n + lane] : -1;
  const bool in = tok >= 0 && tok < a.V;
  const float xt = in ? logit(row, tok) : 0.f;
  int rank = 0;
  if (lane < a.n) {
#pragma unroll 8
    for (int p = 0; p < parts; ++p) rank += ws.ranks[(t * parts + p) * a.n + lane];
  }
#pragma unroll 4
  for (int i = lane; i < total; i += 64) s_keys[i] = ws.keys[t * total + i];
  Part mine = lane < parts ? ws.part[t * parts + lane] : Part{0.f, NOTHING, 0.f, 0.f};
  float top = mine.rest != NOTHING ? mine.top : -INFINITY;
  for (int p = lane + 64; p < parts; p += 64) {
    const Part q = ws.part[t * parts + p];
    if (q.rest != NOTHING) top = fmaxf(top, q.top);
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  const float c = a.scale * ATTN_LOG2E;
  Part stat{about(top), 0.f, 0.f, 0.f};
  float largest_ones = 0.f;  // parts whose own 1 is one of the row's largest
  for (int p = lane; p < parts; p += 64) {
    const Part q = p == lane ? mine : ws.part[t * parts + p];
    if (q.rest == NOTHING) continue;
    if (q.top == stat.top) {
      stat.rest += q.rest;
      stat.t += q.t;
      largest_ones += 1.f;
    } else {
      const float down = fmaxf((q.top - stat.top) * c, -1024.f), f = __builtin_amdgcn_exp2f(down);
      stat.rest += __builtin_fmaf(f, q.rest, f);
      stat.t = __builtin_fmaf(f, __builtin_fmaf(1.f + q.rest, down, q.t), stat.t);
    }
  }
  stat.rest = wave_sum(stat.rest) + (wave_sum(largest_ones) - 1.f);
  stat.t = wave_sum(stat.t);
  const float log_s = log_sum(stat.rest);
  if (lane == 0) row_outputs(a, t, stat, log_s);
  if (lane < a.n) {
    a.logprob[t * a.n + lane] = in ? log_prob(xt, a.scale, stat, log_s) : NAN;
    a.rank[t * a.n + lane] = in ? rank : -1;
  }
  if (a.top == 0) return;
  __syncthreads();
  // The parts' sorted lists are merged: every lane the best of the heads of parts
  // lane, lane + 64, ..; a head that was taken is 0.  Where a lane has one list
  // alone, it also holds the next key of it.
  int place = -1;
  auto find = [&]() {
    uint64_t best = 0;
    place = -1;
    for (int p = lane; p < parts; p += 64)
      for (int j = 0; j < a.top; ++j) {
        const uint64_t k = s_keys[p * a.top + j];
        if (k == 0) continue;
        if (k > best) best = k, place = p * a.top + j;
        break;
      }
    return best;
  };
  const bool single = parts <= 64;
  const int list_end = (lane + 1) * a.top;
  uint64_t head = 0, next = 0, best_key = 0;
  if (single) {
    place = lane * a.top + 1;
    if (lane < parts) head = s_keys[place - 1];
    if (lane < parts && place < list_end) next = s_keys[place];
  } else {
    head = find();
  }
  for (int j = 0; j < a.top; ++j) {
    // the largest value, of equal ones the largest key behind it
    const uint32_t value = wave_max((uint32_t)(head >> 32));
    const uint64_t equal = __ballot((uint32_t)(head >> 32) == value);
    int win = __ffsll((long long)equal) - 1;
    if (equal & (equal - 1)) {
      const uint32_t low = wave_max((uint32_t)(head >> 32) == value ? (uint32_t)head : 0u);
      win = __ffsll((long long)__ballot((uint32_t)(head >> 32) == value && (uint32_t)head == low)) - 1;
    }
    const uint64_t best = (uint64_t)value << 32 | (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)head, win);
    if (lane == j) best_key = best;
    if (lane == win && best) {
      if (single) {
        head = next;
        next = ++place < list_end ? s_keys[place] : 0;
      } else {
        s_keys[place] = 0;
        head = find();
      }
    }
  }
  if (lane < a.top && best_key) {
    a.top_id[t * a.top + lane] = (int32_t)~(uint32_t)best_key;
    a.top_logprob[t * a.top + lane] = log_prob(value_of((uint32_t)(best_key >> 32)), a.scale, stat, log_s);
  }
}

template <class T>
hipError_t launch(const LogprobArgs &a, void *ws, hipStream_t stream) {
  const int ve = 16 / sizeof(T), lead = (int)(reinterpret_cast<uintptr_t>(a.logits) & 15) / (int)sizeof(T);
  const LogprobPlan p = logprob_plan(a.T, a.V, sizeof(T), a.T == 1 || a.ld % ve == 0 ? lead : ve - 1, a.top);
  char *base = static_cast<char *>(ws);
  const LogprobScratch at = logprob_scratch(a.T, p.parts, a.n, a.top);
  static_assert(sizeof(Part) == 16, "scratch of a part");
  const Scratch w{reinterpret_cast<Part *>(base), reinterpret_cast<uint64_t *>(base + at.keys), reinterpret_cast<int32_t *>(base + at.ranks)};
  const int64_t most = rows_of_launch(64 * p.waves * p.parts);
  for (int64_t t0 = 0; t0 < a.T; t0 += most) {
    const unsigned groups = (unsigned)((a.T - t0 < most ? a.T - t0 : most) * p.parts);
#define PART(NV, WAVES) hipLaunchKernelGGL((logprobs_part<T, NV, WAVES>), dim3(groups), dim3(64 * WAVES), 0, stream, a, w, t0, p.parts, p.each)
    if (p.waves == 16) PART(8, 16);
    else if (p.waves == 4) PART(8, 4);
    else if (p.nv == 8) PART(8, 8);
    else if (p.nv == 4) PART(4, 8);
    else if (p.nv == 2) PART(2, 8);
    else PART(1, 8);
#undef PART
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (p.parts == 1) return hipSuccess;
  hipLaunchKernelGGL(logprobs_join<T>, dim3((unsigned)a.T), dim3(64), (size_t)p.parts * a.top * 8, stream, a, w, p.parts);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_logprobs(const LogprobArgs &a, bool bf16, void *ws, hipStream_t stream) {
  return bf16 ? launch<uint16_t>(a, ws, stream) : launch<float>(a, ws, stream);
}

}  // namespace oq
