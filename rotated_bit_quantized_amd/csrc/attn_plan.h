// How one call of oq_attn_prefix is split into items and parts (host only).
#pragma once
#include "oq_internal.h"

namespace oq {

// Page numbers that an item's LDS holds, a single wavefront's and eight
// wavefronts'; a chunk has one page less.
constexpr int NARROW_PAGES = 256, WIDE_PAGES = 512;

// The prefix's or the suffixes' share of the work.
struct PartPlan {
  int suffix;     // 0 prefix (one table, rows of all sequences), 1 suffixes (one sequence per item)
  int wide;       // 1: a workgroup of 8 wavefronts per item, 0: one wavefront
  int tiles;      // row tiles per key head (prefix) or per sequence and key head (suffix)
  int splits;     // chunks of the keys
  int chunk;      // keys per chunk: a multiple of the key tile and of the page (suffixes: the least)
  int part0;      // number of the first part
  int rows;       // B n_q G, rows of one key head
  int swizzle;    // give each XCD a run of items
  int64_t items;
};

// One launch: the workgroups of wide items, then those of one-wavefront items.
struct Launch {
  PartPlan part[2];
  int direct;                           // the only part: no join
  int lead, wide_items, narrow_items, waves;  // workgroups of narrow items before the wide ones; wavefronts of a workgroup
  float c;                              // log2(e) |scale|, or 1 where scale == 0
  uint32_t qxor;                        // on the bits of q pairs: sign of the scale
  int zero;                             // scale == 0: q is taken as 0, NaN where it is not finite
};

struct Plan {
  Launch launch;
  int rows, parts;
  int64_t rows_all;
  bool mixed;
};

Plan plan_for(const AttnArgs &a);

}  // namespace oq
