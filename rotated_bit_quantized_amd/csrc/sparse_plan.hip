#include "sparse_plan.h"

namespace oq {

RoutePlan route_plan(int64_t T, const oq_router &r) {
  RoutePlan p;
  // groups that are all open are none; each group has lanes of its own
  p.l.groups = r.top_groups == r.groups ? 1 : r.groups;
  p.l.lanes = 64 / p.l.groups;
  p.l.each = r.experts / p.l.groups;
  p.l.c = (p.l.each + p.l.lanes - 1) / p.l.lanes;
  p.plain = !r.bias && p.l.groups == 1;
  p.solo = T <= ROUTE_SOLO && p.l.c <= 8;
  // Where logits alone are compared two workgroups fit a CU; with scores and their
  // float64 form one does, and half as many chunks are faster (16384 tokens of 256
  // experts in groups: 43 us, 50 with 512 chunks; logits of 32768 x 128: 32 and 30).
  const int64_t most = p.plain ? ROUTE_CHUNKS : ROUTE_CHUNKS / 2, each = (T + most - 1) / most;
  p.tokens = each < ROUTE_WAVES ? ROUTE_WAVES : (each + ROUTE_WAVES - 1) / ROUTE_WAVES * ROUTE_WAVES;
  if (p.solo) p.tokens = T;
  p.chunks = p.solo ? 1 : (int)((T + p.tokens - 1) / p.tokens);
  return p;
}

size_t route_ws(int64_t T, const oq_router &r) {
  const RoutePlan p = route_plan(T, r);
  return p.solo ? 0 : (size_t)p.chunks * r.experts * 4;
}

LogprobPlan logprob_plan(int64_t T, int V, int bytes, int lead, int top) {
  const int ve = 16 / bytes;
  const int pieces = (V + lead + ve - 1) / ve;
  const int64_t cus = device_cus();
  // Rows that 16 wavefronts can hold and 8 cannot, up to two a CU: one launch (1 x
  // 32000 float32 8.3 us, in 16 parts 9.4; 256 rows 12.5 and 16.2; 256 x 50000 bfloat16 14.7
  // and 18.6, but 32 rows 11.2 and 11.4, 8 11.0 and 10.3, one 10.9 and 9.8).
  if (pieces > 512 * 8 && pieces <= 1024 * 8 && T <= 2 * cus && (bytes == 4 || T >= 32)) return LogprobPlan{16, 8, 1, pieces};
  // Many parts of 4 wavefronts, six workgroups a CU, wait less for each other's threshold
  // than of 8, three a CU (2048 x 131072 bfloat16 127 us and 135, 512 x 16000 10.5 and
  // 12.1); many alternatives cost each part more (20: 153 and 145).
  const int quarter = (pieces + 256 * 8 - 1) / (256 * 8);
  if (top <= 8 && (quarter == 1 ? T >= cus : quarter <= 256 && T * quarter >= 6 * cus))
    return LogprobPlan{4, 8, quarter, (pieces + quarter - 1) / quarter};
  // As many pieces a thread as there are, up to 8, while the parts of all rows still
  // are two workgroups a CU; not more than 256 parts, whose keys the join has in 64 KiB
  // of LDS.
  LogprobPlan p{8, 8, 1, 0};
  for (;; p.nv /= 2) {
    p.parts = (pieces + 512 * p.nv - 1) / (512 * p.nv);
    if (p.nv == 1 || p.parts > 128 || T * p.parts >= 2 * cus) break;
  }
  p.each = (pieces + p.parts - 1) / p.parts;
  return p;
}

LogprobScratch logprob_scratch(int64_t T, int parts, int n, int top) {
  if (parts == 1) return {0, 0, 0};
  auto round16 = [](size_t b) { return (b + 15) & ~(size_t)15; };
  const size_t rows = (size_t)T * parts;
  LogprobScratch s;
  s.keys = rows * 16;
  s.ranks = s.keys + round16(rows * top * 8);
  s.bytes = s.ranks + round16(rows * n * 4);
  return s;
}

size_t logprobs_ws(int64_t T, int V, int n, int top) {
  size_t most = 0;
  for (int bytes = 2; bytes <= 4; bytes += 2)
    for (int lead = 0; lead < 16 / bytes; ++lead) {  // a piece more can choose another plan
      const size_t b = logprob_scratch(T, logprob_plan(T, V, bytes, lead, top).parts, n, top).bytes;
      most = b > most ? b : most;
    }
  return most;
}

}  // namespace oq
