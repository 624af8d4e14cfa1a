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

ExpertPlan expert_plan(int64_t n, int K, int N, int E, bool act) {
  const int64_t cus = device_cus(), outs = act ? N / 2 : N, reached = E < n ? E : n;  // experts with entries, at most
  auto plan = [&](int mt, int ks) {
    const int rows = mt ? 16 * mt : EXPERT_BM, wide = (mt ? 32 * (8 / ks) : EXPERT_BN) / (act ? 2 : 1);
    const int64_t columns = (outs + wide - 1) / wide;
    return ExpertPlan{mt, ks, columns, (columns * (n / rows + reached) + 7) / 8 * 8};
  };
  const int64_t tiles = reached * ((N + EXPERT_BN - 1) / EXPERT_BN);
  // The persistent tiles stream weights as well as anything (16 x 8 entries of 128 experts,
  // 2048 -> 1536: 46.5 us, 5.6 TB/s, gemm_experts_rows 51; 64 x 8 71 and 76; 256 x 8 78 and 98),
  // except where there are too few for half of the CUs: 1 x 8 19.3, rows 11.2; 2 x 2 of 8
  // experts, 4096 -> 7168, 30 and 23; 4 x 2 42 and 50.
  const bool small = K <= 128 * (EXPERT_STAGES - 1);
  if (!small && (tiles > cus / 2 || n > 32 * (int64_t)E)) return plan(0, 1);
  if (n > 16 * (int64_t)E && small) return plan(4, 1);
  // k is split over as many wavefronts as leave the CUs one workgroup each (1 x 4 of 60, 1408 ->
  // 2048: 7.1 us with 8, 8.3 with 4, 15 with 1; 4 x 4: 18.6 with 8, 12.9 with 2)
  const int64_t rows = reached + n / 16, blocks = (outs + (act ? 15 : 31)) / (act ? 16 : 32);
  auto fits = [&](int64_t ks) { return rows * ((blocks * ks + 7) / 8) <= cus + cus / 8; };
  return plan(1, fits(8) ? 8 : fits(4) ? 4 : fits(2) ? 2 : 1);
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
