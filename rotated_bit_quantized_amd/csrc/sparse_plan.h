// How routing, the experts' products and log probabilities divide their work: host code
// of its own, for the launchers, the workspace queries and tests on the CPU.
#pragma once
#include "oq_internal.h"

namespace oq {

// ------------------------------------------------------------------ routing --
constexpr int ROUTE_WAVES = 16;  // of a workgroup; chunks are whole rounds of them
// Up to SOLO tokens one workgroup routes and lists; CHUNKS, LISTS: most workgroups
// of the two launches else.
constexpr int ROUTE_SOLO = 32, ROUTE_CHUNKS = 512, ROUTE_LISTS = 256;

// How a token's experts lie over the lanes of a wavefront.
struct RouteLayout {
  int lanes;  // of a group
  int each;   // experts of a group
  int c;      // experts of a lane, at most 16
  int groups;
};
struct RoutePlan {
  RouteLayout l;
  bool plain;      // the logits alone are compared
  bool solo;       // one workgroup does everything
  int64_t tokens;  // of a chunk
  int chunks;
};
RoutePlan route_plan(int64_t T, const oq_router &r);

// ----------------------------------------------------- experts' products --
// The persistent kernel's tiles: entries x weight rows, and the fewest stages of 128 k of one.
constexpr int EXPERT_BM = 128, EXPERT_BN = 256, EXPERT_STAGES = 4;

struct ExpertPlan {
  int mt, ks;      // 16 mt entries a workgroup, k over ks of its 8 wavefronts; mt 0: persistent tiles
  int64_t columns; // column tiles
  int64_t grid;    // most tiles that n entries of E experts can need, in 8 runs
};
ExpertPlan expert_plan(int64_t n, int K, int N, int E, bool act);

// -------------------------------------------------------- log probabilities --
struct LogprobPlan {
  int waves, nv, parts;  // wavefronts of a workgroup, pieces of 16 bytes a thread, parts of a row
  int each;              // pieces of a part
};
// lead: elements by which rows begin inside a piece; bytes: of an element; top: alternatives.
LogprobPlan logprob_plan(int64_t T, int V, int bytes, int lead, int top);

// Scratch of rows in several parts, in this order, each 16-byte aligned: statistics, keys, ranks.
struct LogprobScratch {
  size_t keys, ranks, bytes;  // places of the last two, and of the end
};
LogprobScratch logprob_scratch(int64_t T, int parts, int n, int top);

}  // namespace oq
