// Routing of tokens to experts and the lists that the experts' products read
// (oq_route).
//
//   s = softmax(l) or sigmoid(l);  c = s + bias, or l itself;  the k largest c of
//   the open groups, their weights;  entries t k + j sorted by expert (stable).
//
// A wavefront takes a token: its experts lie in runs over the lanes, in rising
// order, so that of equal maxima the lowest lane is the lowest index.  Every
// lane sorts its few once; then each choice is one maximum over the lanes' heads
// (six cross-lane steps), one ballot and a shift of the winner's list.  The
// groups' scores come from the same layout, which gives each group lanes of its
// own.  The choices are to be those of the exact scores: float32 scores carry an
// error of less than 2^-19 (1 + |c|), so wherever two neighbours among the
// chosen, the first one left out and the groups at the border are nearer than
// twice that, the token is done again in float64 (one token in some hundreds; a
// choice by the logits themselves compares exactly and never does).
//
// Bound: instructions, some 230 vector and 80 scalar ones a token of 128 experts and 8
// choices, of which the cross-lane maxima are a third: 32768 bfloat16 tokens in 17 us
// (their bytes take 2); for few tokens launches and the length of one token's chain (1
// token 5.4 us, 333 in groups, one a wavefront, 11).
// Lists: a counting sort over at most 512 chunks of tokens.  The routing launch leaves
// each chunk's count of every expert, the second one adds them up (every workgroup
// for itself, four counts a load: that costs less than a third launch; 32768 tokens
// 9 us, 5.3 for few) and writes the entries in order; equal ones of a wavefront find
// their rank by ballots, so no order depends on the time.  Few tokens: one workgroup
// does both.
#include "sparse_plan.h"

namespace oq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int WAVES = ROUTE_WAVES, THREADS = 64 * WAVES;

struct Work {
  RouteArgs a;
  RouteLayout l;
  int64_t tokens;  // of a chunk
  int32_t *hist;   // [chunks][experts]
  int chunks, solo;
};

// Order-preserving whole numbers: larger for larger values, -0 as 0, NaN below
// all numbers (1), above what is not there (0).
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return v != v ? 1u : (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.);
  return v != v ? 1u : (u >> 63) ? ~u : u | 0x8000000000000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k); }

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
  return v > o ? v : o;
}
// the largest over the wavefront, in every lane
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = dpp_max<0xB1, 0xF>(v);   // lane ^ 1
  v = dpp_max<0x4E, 0xF>(v);   // lane ^ 2
  v = dpp_max<0x141, 0xF>(v);  // half mirror of 8
  v = dpp_max<0x140, 0xF>(v);  // mirror of 16
  v = dpp_max<0x142, 0xA>(v);  // last lane of the row before, to rows 1 and 3
  v = dpp_max<0x143, 0xC>(v);  // lane 31 to rows 2 and 3
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
  const uint32_t hi = wave_max((uint32_t)(v >> 32));
  return (uint64_t)hi << 32 | wave_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_other(float v, float none) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(none), __float_as_int(v), CTRL, ROWS, 0xF, false));
}
// the sum over the wavefront and the largest number, in every lane
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_other<0xB1, 0xF>(v, 0.f);
  v += dpp_other<0x4E, 0xF>(v, 0.f);
  v += dpp_other<0x141, 0xF>(v, 0.f);
  v += dpp_other<0x140, 0xF>(v, 0.f);
  v += dpp_other<0x142, 0xA>(v, 0.f);
  v += dpp_other<0x143, 0xC>(v, 0.f);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ float wave_fmax(float v) {
  v = fmaxf(v, dpp_other<0xB1, 0xF>(v, v));
  v = fmaxf(v, dpp_other<0x4E, 0xF>(v, v));
  v = fmaxf(v, dpp_other<0x141, 0xF>(v, v));
  v = fmaxf(v, dpp_other<0x140, 0xF>(v, v));
  v = fmaxf(v, dpp_other<0x142, 0xA>(v, v));
  v = fmaxf(v, dpp_other<0x143, 0xC>(v, v));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ uint32_t read_lane(uint32_t v, int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)v, lane); }
__device__ __forceinline__ uint64_t read_lane(uint64_t v, int lane) {
  return (uint64_t)read_lane((uint32_t)(v >> 32), lane) << 32 | read_lane((uint32_t)v, lane);
}
__device__ __forceinline__ float exp_(float v) { return expf(v); }
__device__ __forceinline__ double exp_(double v) { return exp(v); }
// Whether float32 scores (sums of n of them) may be in the wrong order: each is off by less than
// 2^-19 (1 + |c|), softmax scores by the most, 28 units of 2^-24 (their sum goes over
// at most 16 terms a lane and 6 steps, the exponential and the quotient are 6 more).
__device__ __forceinline__ bool near(float a, float b, float n) { return !(a - b > 0x1p-18f * n * (1.f + fabsf(a) + fabsf(b))); }

// The k choices of a token in F; lane j returns the j-th (others: -1) and, where
// the logits themselves are compared (PLAIN: no bias, no groups), its logit.  x,
// bias: the lane's logits and biases, experts first + i, i < n.
template <int NPL, bool PLAIN, class F>
__device__ __forceinline__ int choose(const float (&x)[NPL], const float (&bias)[NPL], int first, int n, float xmax,
                                      const Work &g, bool &sure, float &logit) {
  const oq_router &r = g.a.r;
  const int lane = threadIdx.x & 63;
  const bool biased = !PLAIN && r.bias != nullptr, grouped = !PLAIN && g.l.groups > 1, sums = grouped && r.group_best == 2;
  using K = decltype(key_of(F()));
  F sc[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) sc[i] = (F)x[i];
  if (biased || sums) {
    if (r.score == OQ_SCORE_SIGMOID) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) sc[i] = F(1) / (F(1) + exp_(-(F)x[i]));
    } else {
      F total = 0;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        sc[i] = exp_((F)x[i] - (F)xmax);
        total += i < n ? sc[i] : F(0);
      }
      total = wave_sum(total);
#pragma unroll
      for (int i = 0; i < NPL; ++i) sc[i] = sc[i] / total;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) sc[i] = biased ? sc[i] + (F)bias[i] : sc[i];
  }
  const bool exact = sizeof(F) == 8 || !biased;
  sure = true;
  bool open = n > 0;
  if (grouped) {
    // the two best of the lane, then of its group (in the group's first lane)
    F b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const F v = i < n && sc[i] == sc[i] ? sc[i] : F(-INFINITY);
      b2 = v > b1 ? b1 : v > b2 ? v : b2;
      b1 = v > b1 ? v : b1;
    }
    const int group = lane / g.l.lanes, sub = lane - group * g.l.lanes;
    for (int o = 1; o < g.l.lanes; o <<= 1) {
      const F o1 = __shfl_down(b1, o), o2 = __shfl_down(b2, o);
      if (sub + o >= g.l.lanes) continue;
      const F low = b1 > o1 ? o1 : b1, up = b2 > o2 ? b2 : o2;
      b2 = low > up ? low : up;
      b1 = b1 > o1 ? b1 : o1;
    }
    const F score = sums ? b1 + b2 : b1;
    const K mine = key_of(score);
    int rank = 0;
    for (int j = 0; j < g.l.groups; ++j) {
      const K other = read_lane(mine, j * g.l.lanes);
      rank += other > mine || (other == mine && j < group);
    }
    const bool head = sub == 0 && group < g.l.groups;
    const uint64_t in = __ballot(head && rank < r.top_groups);
    open = open && (in >> (group * g.l.lanes) & 1);
    if (sizeof(F) == 4 && (biased || sums)) {
      const int last = __ffsll((long long)__ballot(head && rank == r.top_groups - 1)) - 1;
      const int next = __ffsll((long long)__ballot(head && rank == r.top_groups)) - 1;
      if (near((float)__shfl(score, last), (float)__shfl(score, next), 2.f)) sure = false;
    }
    if (!biased && sums) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) sc[i] = (F)x[i];  // inside the groups the logits decide
    }
  }
  // this lane's experts in falling order, equal ones by index: an odd-even sort
  // exchanges neighbours only, and only where the second is larger
  K key[NPL];
  int at[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) key[i] = open && i < n ? key_of(sc[i]) : K(0), at[i] = first + i;
#pragma unroll
  for (int p = 0; p < NPL; ++p) {
#pragma unroll
    for (int i = p & 1; i + 1 < NPL; i += 2) {
      const bool swap = key[i + 1] > key[i];
      const K hi = swap ? key[i + 1] : key[i], lo = swap ? key[i] : key[i + 1];
      const int hat = swap ? at[i + 1] : at[i], lat = swap ? at[i] : at[i + 1];
      key[i] = hi, key[i + 1] = lo, at[i] = hat, at[i + 1] = lat;
    }
  }
  int chosen = -1;
  K before = 0;
  for (int j = 0; j <= r.k; ++j) {
    if (j == r.k && exact) break;  // the first one left out, to see how near it is
    const K m = wave_max(key[0]);
    if (sizeof(F) == 4 && !exact && j && m && near(value_of((uint32_t)before), value_of((uint32_t)m), 1.f)) sure = false;
    if (j == r.k) break;
    before = m;
    const int win = __ffsll((long long)__ballot(key[0] == m)) - 1;
    const int id = __builtin_amdgcn_readlane(at[0], win);
    if (lane == j) {
      chosen = id;
      if constexpr (PLAIN) logit = value_of(m);
    }
    if (lane == win) {
#pragma unroll
      for (int i = 0; i + 1 < NPL; ++i) key[i] = key[i + 1], at[i] = at[i + 1];
      key[NPL - 1] = 0;
    }
  }
  return chosen;
}

// choose() where 16-bit logits alone are compared: value and index share a word, the
// index falling, so no two keys are equal and the largest one says everything.
template <int NPL>
__device__ __forceinline__ int choose_packed(const float (&x)[NPL], int first, int n, int k, float &logit) {
  const int lane = threadIdx.x & 63;
  uint32_t key[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) key[i] = i < n ? (key_of(x[i]) & 0xFFFF0000u) | (uint32_t)(0xFFFF - first - i) : 0u;
#pragma unroll
  for (int p = 0; p < NPL; ++p) {
#pragma unroll
    for (int i = p & 1; i + 1 < NPL; i += 2) {
      const uint32_t a = key[i], b = key[i + 1];
      key[i] = a > b ? a : b, key[i + 1] = a > b ? b : a;
    }
  }
  uint32_t mine = 0;
  for (int j = 0; j < k; ++j) {
    const uint32_t m = wave_max(key[0]);
    mine = lane == j ? m : mine;
    if (key[0] == m) {
#pragma unroll
      for (int i = 0; i + 1 < NPL; ++i) key[i] = key[i + 1];
      key[NPL - 1] = 0;
    }
  }
  logit = __uint_as_float((mine >> 31) ? mine & 0x7FFF0000u : ~mine & 0xFFFF0000u);  // NaN, whose value is 0, is one again
  return 0xFFFF - (int)(mine & 0xFFFFu);
}

// The weight of the lane's chosen expert (lanes below k).
__device__ __forceinline__ float weight(float x, bool mine, float xmax, float total, bool nan, const oq_router &r) {
  float s = 0.f;
  if (r.score == OQ_SCORE_SOFTMAX) {
    // among themselves the chosen are a softmax of their own: no scores that
    // vanish in float32
    const float top = r.renorm ? wave_fmax(mine ? x : -INFINITY) : xmax;
    s = mine ? expf(x - top) : 0.f;
    if (nan) s = NAN;
    total = r.renorm ? wave_sum(s) : total;
    return r.factor * (s / total);
  }
  // sigmoids of which all are small, scaled by the largest: e^(x - low) / (1 + e^x)
  const float low = r.renorm ? fminf(0.f, wave_fmax(mine ? x : -INFINITY)) : 0.f;
  if (mine) s = x >= 0.f ? 1.f / (1.f + expf(-x)) : expf(x - low) / (1.f + expf(x));
  return r.factor * (r.renorm ? s / wave_sum(s) : s);
}

template <int NPL, int W, bool PLAIN, class T>
__device__ __forceinline__ void route_tokens(const Work &g, int64_t t0, int64_t t1, int *hist) {
  const RouteArgs &a = g.a;
  const oq_router &r = a.r;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // a token's addresses are scalar
  const int group = lane / g.l.lanes, sub = lane - group * g.l.lanes;
  const int first = group * g.l.each + sub * g.l.c;
  int n = g.l.each - sub * g.l.c;
  n = group >= g.l.groups || n < 0 ? 0 : n < g.l.c ? n : g.l.c;
  float bias[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) bias[i] = r.bias && i < n ? r.bias[first + i] : 0.f;
  auto load = [&](float (&x)[NPL], int64_t t) {
    const T *row = static_cast<const T *>(a.logits) + t * a.ld + first;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      x[i] = -INFINITY;
      if (i < n) {
        if constexpr (sizeof(T) == 2) x[i] = __uint_as_float((uint32_t)row[i] << 16);
        else x[i] = row[i];
      }
    }
  };
  float x[NPL], xn[NPL];
  if (t0 + wave < t1) load(x, t0 + wave);
  for (int64_t t = t0 + wave; t < t1; t += W) {
    if (t + W < t1) load(xn, t + W);  // the next token's under this one's choices
    int id = -1;
    float w = 0.f;
    if (!a.mask || a.mask[t]) {
      const bool softmax = r.score == OQ_SCORE_SOFTMAX;
      const bool scores = !PLAIN && (r.bias || (g.l.groups > 1 && r.group_best == 2));
      float xmax = -INFINITY, total = 0.f;
      bool nan = false;
      if (softmax) {
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          xmax = fmaxf(xmax, x[i]);
          nan = nan || (PLAIN ? x[i] != x[i] : !(x[i] < INFINITY));  // a plain choice takes an infinity itself
        }
        nan = __any(nan);
        if (scores || !r.renorm) xmax = wave_fmax(xmax);
        if (!r.renorm) {
#pragma unroll
          for (int i = 0; i < NPL; ++i) total += i < n ? expf(x[i] - xmax) : 0.f;
          total = wave_sum(total);
        }
      }
      bool sure;
      float chosen = 0.f;
      const bool mine = lane < r.k;
      if constexpr (PLAIN && sizeof(T) == 2) id = choose_packed<NPL>(x, first, n, r.k, chosen);
      else id = choose<NPL, PLAIN, float>(x, bias, first, n, xmax, g, sure, chosen);
      if constexpr (!PLAIN) {
        if (!sure) id = choose<NPL, PLAIN, double>(x, bias, first, n, xmax, g, sure, chosen);
        if (mine) {
          const T v = static_cast<const T *>(a.logits)[t * a.ld + id];
          if constexpr (sizeof(T) == 2) chosen = __uint_as_float((uint32_t)v << 16);
          else chosen = v;
        }
      }
      w = weight(chosen, mine, xmax, total, nan, r);
    }
    if (lane < r.k) {
      a.ids[t * r.k + lane] = id;
      a.weights[t * r.k + lane] = w;
      if (hist && id >= 0) atomicAdd(hist + id, 1);
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) x[i] = xn[i];
  }
}

// Exclusive sums of v over the threads of the workgroup and the sum of all.
__device__ __forceinline__ int scan_block(int v, int *wave_sums, int &all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(s, o);
    if (lane >= o) s += u;
  }
  if (lane == 63) wave_sums[wave] = s;
  __syncthreads();
  int below = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    below += w < wave ? wave_sums[w] : 0;
    all += wave_sums[w];
  }
  __syncthreads();
  return below + s - v;
}

// Entries i0 .. i1 - 1 to their places: expert e's go to base[e], base[e] + 1, ..
// count: [WAVES][E] in LDS.
__device__ __forceinline__ void scatter(const RouteArgs &a, int64_t i0, int64_t i1, int *base, uint16_t *count) {
  const int E = a.r.experts, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int bits = 32 - __clz(E);  // E itself stands for no expert
  for (int64_t at = i0; at < i1; at += THREADS) {
    for (int j = threadIdx.x; j < WAVES * E; j += THREADS) count[j] = 0;
    __syncthreads();
    const int64_t i = at + threadIdx.x;
    const int id = i < i1 ? a.ids[i] : -1;
    const int tag = id < 0 ? E : id;
    uint64_t same = ~0ull;
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot(tag >> b & 1);
      same &= tag >> b & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    if (id >= 0 && rank == 0) count[wave * E + id] = (uint16_t)__popcll(same);
    __syncthreads();
    int sum = 0;  // thread e: the entries of expert e in the wavefronts before
    if (threadIdx.x < E) {
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const int c = count[w * E + threadIdx.x];
        count[w * E + threadIdx.x] = (uint16_t)sum;
        sum += c;
      }
    }
    __syncthreads();
    if (id >= 0) a.order[base[id] + count[wave * E + id] + rank] = (int32_t)i;
    __syncthreads();
    if (threadIdx.x < E) base[threadIdx.x] += sum;
  }
}

__device__ __forceinline__ void fill_tail(const RouteArgs &a, int64_t i0, int64_t i1, int64_t listed) {
  for (int64_t i = (i0 > listed ? i0 : listed) + threadIdx.x; i < i1; i += THREADS) a.order[i] = -1;
}

// W wavefronts: 16, or 8 where a lane's lists need the registers of two.
template <int NPL, int W, bool PLAIN, class T>
__global__ void __launch_bounds__(64 * W) route_kernel(const Work g) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  int *hist = reinterpret_cast<int *>(smem);
  const RouteArgs &a = g.a;
  const int E = a.r.experts;
  const bool lists = a.offsets != nullptr;
  if (lists) {
    for (int e = threadIdx.x; e < E; e += 64 * W) hist[e] = 0;
    __syncthreads();
  }
  const int64_t t0 = blockIdx.x * g.tokens, t1 = t0 + g.tokens < a.T ? t0 + g.tokens : a.T;
  route_tokens<NPL, W, PLAIN, T>(g, t0, t1, lists ? hist : nullptr);
  if (!lists) return;
  __syncthreads();
  if (W < WAVES || !g.solo) {
    for (int e = threadIdx.x; e < E; e += 64 * W) g.hist[(int64_t)blockIdx.x * E + e] = hist[e];
    return;
  }
  if constexpr (W == WAVES) {
    __shared__ int wave_sums[WAVES];
    int all;
    const int below = scan_block(threadIdx.x < E ? hist[threadIdx.x] : 0, wave_sums, all);
    if (threadIdx.x < E) hist[threadIdx.x] = a.offsets[threadIdx.x] = below;
    if (threadIdx.x == 0) a.offsets[E] = all;
    __syncthreads();
    scatter(a, 0, a.T * a.r.k, hist, reinterpret_cast<uint16_t *>(hist + E));
    fill_tail(a, 0, a.T * a.r.k, all);
  }
}

__global__ void __launch_bounds__(THREADS) route_lists_kernel(const Work g) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  __shared__ int wave_sums[WAVES];
  const RouteArgs &a = g.a;
  // this workgroup's chunks; every one of them before it costs a row of counts
  const int E = a.r.experts, chunks = g.chunks, share = (chunks + (int)gridDim.x - 1) / (int)gridDim.x;
  const int chunk = blockIdx.x * share;
  int *base = reinterpret_cast<int *>(smem), *total = base + E;
  if (threadIdx.x < E) base[threadIdx.x] = total[threadIdx.x] = 0;
  __syncthreads();
  // rows of counts in turn over groups of threads, four counts a load where they allow
  auto add_rows = [&](auto load, int cols, int width) {
    const int rows = THREADS / cols < 64 ? THREADS / cols : 64;  // more would meet in the same few sums
    const int row = threadIdx.x / cols, col = threadIdx.x - row * cols;
    if (row >= rows) return;
    i32x4 before = {0, 0, 0, 0}, sum = {0, 0, 0, 0};
#pragma unroll 16
    for (int c = row; c < chunks; c += rows) {
      const i32x4 v = load((int64_t)c * E + col * width);
      before += c < chunk ? v : (i32x4){0, 0, 0, 0};
      sum += v;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= width) continue;
      atomicAdd(base + col * width + j, before[j]);
      atomicAdd(total + col * width + j, sum[j]);
    }
  };
  if (E % 4 == 0) add_rows([&](int64_t i) { return *reinterpret_cast<const i32x4 *>(g.hist + i); }, E / 4, 4);
  else add_rows([&](int64_t i) { return (i32x4){g.hist[i], 0, 0, 0}; }, E, 1);
  __syncthreads();
  int all;
  const int start = scan_block(threadIdx.x < E ? total[threadIdx.x] : 0, wave_sums, all);
  if (threadIdx.x < E) {
    base[threadIdx.x] += start;
    if (blockIdx.x == 0) a.offsets[threadIdx.x] = start;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[E] = all;
  __syncthreads();
  const int64_t t0 = chunk * g.tokens < a.T ? chunk * g.tokens : a.T, t1 = t0 + share * g.tokens < a.T ? t0 + share * g.tokens : a.T;
  scatter(a, t0 * a.r.k, t1 * a.r.k, base, reinterpret_cast<uint16_t *>(total + E));
  fill_tail(a, t0 * a.r.k, t1 * a.r.k, all);
}

template <bool PLAIN, class T>
hipError_t launch(const Work &g, unsigned chunks, hipStream_t stream) {
  const int E = g.a.r.experts;
  const size_t lds = g.a.offsets ? (size_t)E * 4 + (g.solo ? (size_t)E * 2 * WAVES : 0) : 0;
#define ROUTE(NPL, W) hipLaunchKernelGGL((route_kernel<NPL, W, PLAIN, T>), dim3(chunks), dim3(64 * W), lds, stream, g)
  if (g.l.c <= 1) ROUTE(1, 16);
  else if (g.l.c <= 2) ROUTE(2, 16);
  else if (g.l.c <= 4) ROUTE(4, 16);
  else if (g.l.c <= 8) ROUTE(8, 16);
  else ROUTE(16, 8);
#undef ROUTE
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs &a, bool bf16, void *ws, hipStream_t stream) {
  const RoutePlan p = route_plan(a.T, a.r);
  const Work g{a, p.l, p.tokens, static_cast<int32_t *>(ws), p.chunks, p.solo && a.offsets};
  if (a.T > 0 || g.solo) {
    const hipError_t e = p.plain ? bf16 ? launch<true, uint16_t>(g, p.chunks, stream) : launch<true, float>(g, p.chunks, stream)
                         : bf16  ? launch<false, uint16_t>(g, p.chunks, stream)
                                 : launch<false, float>(g, p.chunks, stream);
    if (e != hipSuccess) return e;
  }
  if (!a.offsets || g.solo) return hipSuccess;
  const size_t lds = (size_t)a.r.experts * (8 + 2 * WAVES);
  const int lists = p.chunks < 1 ? 1 : p.chunks < ROUTE_LISTS ? p.chunks : ROUTE_LISTS;  // without tokens the lists are empty
  hipLaunchKernelGGL(route_lists_kernel, dim3(lists), dim3(THREADS), lds, stream, g);
  return hipGetLastError();
}

}  // namespace oq
