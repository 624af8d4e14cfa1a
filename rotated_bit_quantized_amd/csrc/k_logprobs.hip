// Log probabilities, ranks, entropy and best alternatives of rows of logits
// (oq_logprobs).
//
//   z = scale log2(e) x - M,  s = sum 2^z,  t = sum 2^z z     (M: the largest)
//   lse = ln2 (M + log2 s),  log p = ln2 (z - log2 s),  entropy = ln2 (log2 s - t / s)
//
// Bound: HBM, one pass over the logits; some 12 vector instructions an element
// are near that.  A workgroup takes a part of a row, its pieces of 16 bytes all
// in flight at once and held in registers: the maximum is known before the first
// exponential, so nothing is rescaled, and what comes after it (ranks, best
// alternatives) reads registers.
//
// Alternatives: the `top`-th largest of 64 maxima (over the threads of one lane
// number) is a threshold that at least `top` elements reach and hardly more do;
// those go to a list in LDS and are ranked there as whole numbers (value, then
// falling index), so ties never depend on the time.  Rows in which more than the
// list holds reach the threshold (many equal values, or the best ones all in one
// lane's places) get the exact value by bisection, and of values equal to it the
// first ones in order.
//
// Rows of several parts leave statistics and sorted candidates for a second
// launch, a wavefront a row.
#include "oq_internal.h"

namespace oq {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int WAVES = 8, THREADS = 64 * WAVES, LIST = 512;
constexpr float LN2 = 0.693147180559945309417f;

// What is known of a row or a part of it: sums over 2^(z(x)).
struct Part {
  float top, m, s, t;  // the largest logit, m = RN(top scale log2(e))
};

// z of a logit.  Where m passes float32 (logits next to the type's ends: a mask of
// the lowest value) the difference is formed first; else in one step, whose only
// rounding is that of z.
__device__ __forceinline__ float z_of(float x, float c, const Part &r) {
  return fabsf(r.m) < INFINITY ? __builtin_fmaf(x, c, -r.m) : (x - r.top) * c;
}
// The reference of logits of which `top` is the largest; of nothing but -inf any does.
__device__ __forceinline__ Part about(float top, float c) {
  const float ref = top == -INFINITY ? 0.f : top;
  return Part{ref, ref * c, 0.f, 0.f};
}

struct Plan {
  int nv, parts;
};

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
__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    const uint64_t w = (uint64_t)__shfl_xor((unsigned long long)v, o);
    v = v > w ? v : w;
  }
  return v;
}

template <class T>
__device__ __forceinline__ float logit(const T *row, int i) {
  if constexpr (sizeof(T) == 2) return __uint_as_float((uint32_t)row[i] << 16);
  else return row[i];
}

// What a row's statistics say of a logit and of the row.
__device__ __forceinline__ float log_prob(float x, float scale, const Part &r) {
  const float z = z_of(x, scale * ATTN_LOG2E, r), log_s = log2f(r.s);
  if (z == -INFINITY && x > -INFINITY && r.top < INFINITY) return (x - r.top) * scale;  // in units of log 2 it passes float32
  return (z - log_s) * LN2;
}
__device__ __forceinline__ void row_outputs(const LogprobArgs &a, int64_t t, const Part &r) {
  const float log_s = log2f(r.s);
  if (a.lse) a.lse[t] = fabsf(r.m) < INFINITY ? (r.m + log_s) * LN2 : __builtin_fmaf(r.top, a.scale, log_s * LN2);
  if (a.entropy) a.entropy[t] = (log_s - r.t / r.s) * LN2;
}
template <class T>
__device__ __forceinline__ void token_outputs(const LogprobArgs &a, const T *row, int64_t t, int i, const Part &r, int rank) {
  const int tok = a.tokens[t * a.n + i];
  const bool in = tok >= 0 && tok < a.V;
  a.logprob[t * a.n + i] = in ? log_prob(logit(row, tok), a.scale, r) : NAN;
  a.rank[t * a.n + i] = in ? rank : -1;
}

template <class T, int NV>
__global__ void __launch_bounds__(THREADS) logprobs_part(const LogprobArgs a, const Scratch ws, const int parts) {
  constexpr int VE = 16 / sizeof(T);  // elements of a piece
  __shared__ uint32_t s_max[WAVES * 64];
  __shared__ float s_sum[2 * WAVES];
  __shared__ uint64_t s_list[LIST];
  __shared__ int s_rank[64];
  __shared__ int s_count[2];
  __shared__ uint32_t s_limit;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.x / parts;
  const int part = blockIdx.x - (int)(t * parts);
  const T *row = static_cast<const T *>(a.logits) + t * a.ld;
  // pieces lie on 16-byte boundaries: the first one may begin before the row
  const int lead = (int)(reinterpret_cast<uintptr_t>(row) & 15) / (int)sizeof(T);
  const int first = (part * NV * THREADS + (int)threadIdx.x) * VE - lead;  // element of this thread's first piece
  constexpr int STEP = THREADS * VE;
  constexpr uint32_t NONE = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;  // -inf
  u32x4 raw[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = first + v * STEP;
    raw[v] = (u32x4){NONE, NONE, NONE, NONE};
    if (i >= 0 && i + VE <= a.V) {
      raw[v] = *reinterpret_cast<const u32x4 *>(row + i);
    } else if (i + VE > 0 && i < a.V) {  // a piece that the row fills in part
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        if (i + j < 0 || i + j >= a.V) continue;
        if constexpr (sizeof(T) == 2) {
          const uint32_t w = raw[v][j / 2], e = row[i + j];
          raw[v][j / 2] = j & 1 ? (w & 0xFFFFu) | e << 16 : (w & 0xFFFF0000u) | e;
        } else {
          raw[v][j] = __float_as_uint(row[i + j]);
        }
      }
    }
  }
  auto at = [&](int v, int j) {
    if constexpr (sizeof(T) == 2) return j & 1 ? bf16_hi(raw[v][j / 2]) : bf16_lo(raw[v][j / 2]);
    else return __uint_as_float(raw[v][j]);
  };
  // what was unpacked for one pass over the registers is not kept for the next
  auto forget = [&]() {
#pragma unroll
    for (int v = 0; v < NV; ++v) asm volatile("" : "+v"(raw[v]));
  };
  if (threadIdx.x < 64) s_rank[threadIdx.x] = 0;
  if (threadIdx.x < 2) s_count[threadIdx.x] = 0;

  float mine = -INFINITY;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int j = 0; j < VE; ++j) mine = fmaxf(mine, at(v, j));  // passes NaN over
  s_max[threadIdx.x] = order_of(mine);
  __syncthreads();
  uint32_t group = 0;  // the largest over the threads of this lane number
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    const uint32_t o = s_max[64 * w + lane];
    group = o > group ? o : group;
  }
  const float top = value_of(wave_max(group)), c = a.scale * ATTN_LOG2E;
  Part stat = about(top, c);

  float s = 0.f, sum_t = 0.f;
  auto sums = [&](auto z_at) {
    forget();
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float z = z_at(at(v, j)), e = __builtin_amdgcn_exp2f(z);
        s += e;
        sum_t = __builtin_fmaf(e, fmaxf(z, -1024.f), sum_t);  // 2^-inf takes no part
      }
  };
  if (fabsf(stat.m) < INFINITY) sums([&](float x) { return __builtin_fmaf(x, c, -stat.m); });
  else sums([&](float x) { return (x - stat.top) * c; });
  s = wave_sum(s);
  sum_t = wave_sum(sum_t);
  if (lane == 0) s_sum[wave] = s, s_sum[WAVES + wave] = sum_t;

  // ranks: elements above the token's, and equal ones before it.  A piece before
  // the token counts from its value on, one behind it from the next value on.
  for (int i = 0; i < a.n; ++i) {
    const int tok = a.tokens[t * a.n + i];
    if (tok < 0 || tok >= a.V) continue;
    const float xt = logit(row, tok);
    int count = 0;
    forget();
    if (xt > -INFINITY) {
      const float above = value_of(order_of(xt) + 1);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int i0 = first + v * STEP;
        const float limit = i0 + VE <= tok ? xt : above;
#pragma unroll
        for (int j = 0; j < VE; ++j) count += __popcll(__ballot(at(v, j) >= limit));
        if (i0 <= tok && tok < i0 + VE) {  // one thread of the row: equal ones in the token's own piece
          int equal = 0;
#pragma unroll
          for (int j = 0; j < VE; ++j) equal += i0 + j < tok && at(v, j) == xt;
          atomicAdd(s_rank + i, equal);
        }
      }
    } else {  // -inf or NaN: places outside the row would count too
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const int at_i = first + v * STEP + j;
          const float x = at(v, j);
          const uint32_t o = order_of(x), ot = order_of(xt);
          count += __popcll(__ballot(at_i >= 0 && at_i < a.V && (o > ot || (o == ot && at_i < tok))));
        }
    }
    if (lane == 0 && count) atomicAdd(s_rank + i, count);
  }

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
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WAVES; ++w) stat.s += s_sum[w], stat.t += s_sum[WAVES + w];

  if (a.top > 0) {
    const uint32_t lowest = order_of(-INFINITY);
    uint32_t limit = s_limit;
    auto add = [&](float x, int i) {
      const int n = atomicAdd(s_count, 1);
      if (n < LIST) s_list[n] = key_of(x, i);
    };
    auto collect = [&](uint32_t from) {  // every number of order `from` on, from > lowest
      const float v0 = value_of(from);
      forget();
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < VE; ++j)
          if (at(v, j) >= v0) add(at(v, j), first + v * STEP + j);
    };
    auto count_from = [&](uint32_t from, int slot) {  // how many numbers of order `from` on, from > lowest
      const float v0 = value_of(from);
      forget();
      int count = 0;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < VE; ++j) count += __popcll(__ballot(at(v, j) >= v0));
      __syncthreads();
      if (threadIdx.x == 0) s_count[slot] = 0;
      __syncthreads();
      if (lane == 0) atomicAdd(s_count + slot, count);
      __syncthreads();
      return s_count[slot];
    };
    // the first `want` elements of order o in this wavefront, by index
    auto collect_first = [&](uint32_t o, int want) {
      for (int v = 0; v < NV && want > 0; ++v) {
        uint32_t hit = 0;
        forget();
#pragma unroll
        for (int w = 0; w < NV; ++w)  // raw[] stays in registers
          if (w == v) {
#pragma unroll
            for (int j = 0; j < VE; ++j) {
              const int i = first + w * STEP + j;
              hit |= (uint32_t)(i >= 0 && i < a.V && order_of(at(w, j)) == o) << j;
            }
          }
        int before = 0, all = 0;
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const uint64_t b = __ballot(hit >> j & 1);
          before += __popcll(b & ((1ull << lane) - 1));
          all += __popcll(b);
        }
        const float x = value_of(o);
#pragma unroll
        for (int j = 0; j < VE; ++j)
          if (hit >> j & 1 && before++ < want) add(x, first + v * STEP + j);
        want -= all;
      }
    };
    bool listed = false;
    if (limit > lowest) {
      collect(limit);
      __syncthreads();
      listed = s_count[0] <= LIST;
      __syncthreads();
    }
    if (!listed) {
      // too many: the exact top-th value, unless fewer are above the limit
      int above = count_from(limit + 1, 1);
      if (above >= a.top) {
        uint32_t lo = limit + 1, hi = order_of(top) + 1;  // count(lo) >= top, count(hi) = 0
        while (hi - lo > 1) {
          const uint32_t mid = lo + (hi - lo) / 2;
          if (count_from(mid, 1) >= a.top) lo = mid;
          else hi = mid;
        }
        limit = lo;
        above = count_from(limit + 1, 1);
      }
      __syncthreads();
      if (threadIdx.x == 0) s_count[0] = 0;
      __syncthreads();
      if (above > 0) collect(limit + 1);
      collect_first(limit, a.top - above);
      __syncthreads();
      const int n = s_count[0];
      __syncthreads();
      if (limit == lowest && n < a.top) collect_first(1, a.top - n);  // fewer numbers than that: NaN
      __syncthreads();
    }
    const int n = s_count[0];
    const uint64_t key = (int)threadIdx.x < n ? s_list[threadIdx.x] : 0;
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += s_list[j] > key;
    if (parts == 1) {
      if ((int)threadIdx.x < n && rank < a.top) {
        a.top_id[t * a.top + rank] = (int32_t)~(uint32_t)key;
        a.top_logprob[t * a.top + rank] = log_prob(value_of((uint32_t)(key >> 32)), a.scale, stat);
      }
    } else {
      uint64_t *keys = ws.keys + ((int64_t)t * parts + part) * a.top;
      if ((int)threadIdx.x < n && rank < a.top) keys[rank] = key;
      if ((int)threadIdx.x >= n && (int)threadIdx.x < a.top) keys[threadIdx.x] = 0;
    }
  }
  if (parts == 1) {
    if (threadIdx.x == 0) row_outputs(a, t, stat);
    if ((int)threadIdx.x < a.n) token_outputs(a, row, t, threadIdx.x, stat, s_rank[threadIdx.x]);
  } else {
    if (threadIdx.x == 0) ws.part[t * parts + part] = stat;
    if ((int)threadIdx.x < a.n) ws.ranks[(t * parts + part) * a.n + threadIdx.x] = s_rank[threadIdx.x];
  }
}

template <class T>
__global__ void __launch_bounds__(64) logprobs_join(const LogprobArgs a, const Scratch ws, const int parts) {
  extern __shared__ uint64_t s_keys[];  // [parts][top]
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x;
  const T *row = static_cast<const T *>(a.logits) + t * a.ld;
  const int total = parts * a.top;
  for (int i = lane; i < total; i += 64) s_keys[i] = ws.keys[t * total + i];
  // parts of nothing but -inf (s = 0) have no maximum
  float top = -INFINITY;
  for (int p = lane; p < parts; p += 64) {
    const Part q = ws.part[t * parts + p];
    if (q.s != 0.f) top = fmaxf(top, q.top);
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  const float c = a.scale * ATTN_LOG2E;
  Part stat = about(top, c);
  for (int p = lane; p < parts; p += 64) {
    const Part q = ws.part[t * parts + p];
    if (q.s == 0.f) continue;
    const bool far = !(fabsf(q.m) < INFINITY && fabsf(stat.m) < INFINITY);
    const float down = fmaxf(far ? (q.top - stat.top) * c : q.m - stat.m, -1024.f), f = __builtin_amdgcn_exp2f(down);
    stat.s = __builtin_fmaf(f, q.s, stat.s);
    stat.t = __builtin_fmaf(f, __builtin_fmaf(q.s, down, q.t), stat.t);
  }
  stat.s = wave_sum(stat.s);
  stat.t = wave_sum(stat.t);
  if (lane == 0) row_outputs(a, t, stat);
  for (int i = lane; i < a.n; i += 64) {
    int rank = 0;
    for (int p = 0; p < parts; ++p) rank += ws.ranks[(t * parts + p) * a.n + i];
    token_outputs(a, row, t, i, stat, rank);
  }
  if (a.top == 0) return;
  __syncthreads();
  // the parts' sorted lists are merged: every lane the best of its parts' heads,
  // packed behind the key's index as nothing but the place in LDS
  int mine = -1;  // place of the best head of parts lane, lane + 64, ..
  auto find = [&]() {
    uint64_t best = 0;
    mine = -1;
    for (int p = lane; p < parts; p += 64)
      for (int j = 0; j < a.top; ++j) {  // heads that were taken are 0
        const uint64_t k = s_keys[p * a.top + j];
        if (k == 0) continue;
        if (k > best) best = k, mine = p * a.top + j;
        break;
      }
    return best;
  };
  uint64_t head = find();
  for (int j = 0; j < a.top; ++j) {
    const uint64_t best = wave_max64(head);
    if (head == best && best) {
      a.top_id[t * a.top + j] = (int32_t)~(uint32_t)best;
      a.top_logprob[t * a.top + j] = log_prob(value_of((uint32_t)(best >> 32)), a.scale, stat);
      s_keys[mine] = 0;
      head = find();
    }
  }
}

// Pieces a thread and parts a row: as many pieces as there are, up to 8, while the parts of
// all rows still are two workgroups a CU.
Plan plan_for(int64_t T, int V, int bytes) {
  const int ve = 16 / bytes;
  const int64_t pieces = ((int64_t)V + 2 * (ve - 1)) / ve;  // a row that begins inside a piece has one more
  Plan p{8, 1};
  for (;; p.nv /= 2) {
    p.parts = (int)((pieces + (int64_t)THREADS * p.nv - 1) / ((int64_t)THREADS * p.nv));
    if (p.nv == 1 || T * p.parts >= 2 * device_cus()) return p;
  }
}

size_t round16(size_t n) { return (n + 15) & ~(size_t)15; }
size_t scratch_bytes(int64_t T, int parts, int n, int top) {
  if (parts == 1) return 0;
  const size_t rows = (size_t)T * parts;
  return rows * sizeof(Part) + round16(rows * top * 8) + round16(rows * n * 4);
}

template <class T>
hipError_t launch(const LogprobArgs &a, void *ws, hipStream_t stream) {
  const Plan p = plan_for(a.T, a.V, sizeof(T));
  const size_t rows = (size_t)a.T * p.parts;
  if (rows > 0x7fffffff) return hipErrorInvalidConfiguration;
  char *base = static_cast<char *>(ws);
  const Scratch w{reinterpret_cast<Part *>(base), reinterpret_cast<uint64_t *>(base + rows * sizeof(Part)),
                  reinterpret_cast<int32_t *>(base + rows * sizeof(Part) + round16(rows * a.top * 8))};
#define PART(NV) hipLaunchKernelGGL((logprobs_part<T, NV>), dim3((unsigned)rows), dim3(THREADS), 0, stream, a, w, p.parts)
  if (p.nv == 8) PART(8);
  else if (p.nv == 4) PART(4);
  else if (p.nv == 2) PART(2);
  else PART(1);
#undef PART
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.parts == 1) return e;
  hipLaunchKernelGGL(logprobs_join<T>, dim3((unsigned)a.T), dim3(64), (size_t)p.parts * a.top * 8, stream, a, w, p.parts);
  return hipGetLastError();
}

}  // namespace

size_t logprobs_ws(int64_t T, int V, int n, int top) {
  const size_t b = scratch_bytes(T, plan_for(T, V, 2).parts, n, top), f = scratch_bytes(T, plan_for(T, V, 4).parts, n, top);
  return b > f ? b : f;
}

hipError_t launch_logprobs(const LogprobArgs &a, bool bf16, void *ws, hipStream_t stream) {
  return bf16 ? launch<uint16_t>(a, ws, stream) : launch<float>(a, ws, stream);
}

}  // namespace oq
