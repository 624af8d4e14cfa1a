// The plan of oq_attn_prefix: which rows and keys make an item, how many parts
// the keys have, what their partial results take (host code; the measurements
// behind each rule stand at the rule).
#include "attn_plan.h"

namespace oq {

static int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

Plan plan_for(const AttnArgs &a) {
  Plan p{};
  const int G = a.heads_q / a.kv.heads;
  p.rows = a.B * a.n_q * G;
  p.rows_all = (int64_t)p.rows * a.kv.heads;
  const int64_t cus = device_cus();
  int64_t keys[2], groups[2];
  double work[2];
  for (int s = 0; s < 2; ++s) {
    PartPlan &q = p.launch.part[s];
    keys[s] = a.kv.pages == 0 ? 0 : s ? (int64_t)a.table_ld * a.kv.page : a.prefix_len;
    const int group_rows = s ? a.n_q * G : p.rows;
    q.suffix = s;
    q.rows = p.rows;
    // Wavefronts on their own read a key once per 32 rows, but start at once and
    // go to every CU; eight that share keys through LDS read them once per 256
    // rows.  Single ones up to 64 rows, or where 16 a CU with 64 keys each are
    // enough.  Single against shared: 96 rows of 8 heads over 16384
    // keys 40.9 us (33.4), over 2000 15.9 (21.1); 160 of 8 over 8000 31.7 (28.4);
    // 256 of 4 over 2000 17.7 (23.9).
    const int64_t singles = (int64_t)((group_rows + 31) / 32) * a.kv.heads * (s ? a.B : 1) * ((keys[s] + 63) / 64);
    q.wide = group_rows > 64 && singles > 16 * cus;
    q.tiles = (group_rows + (q.wide ? 255 : 31)) / (q.wide ? 256 : 32);
    groups[s] = (int64_t)q.tiles * a.kv.heads * (s ? a.B : 1);
    // CU microseconds, as measured: 2.0 (d 128) or 1.1 (d 64) for 64 keys of a
    // wide item, 4 and 1.9 or 1.2 per 32 keys for eight single wavefronts (used
    // to share the CUs below); suffixes are taken to fill half of their tables
    const double k = s ? 0.5 * (double)keys[s] : (double)keys[s];
    work[s] = keys[s] == 0 ? 0
              : q.wide     ? (double)groups[s] * k / 64 * (a.kv.d == 128 ? 2.0 : 1.1)
                           : (double)groups[s] / 8 * (4 + k / 32 * (a.kv.d == 128 ? 1.9 : 1.2));
  }
  // Chunks that give every CU a workgroup, or eight single wavefronts.  Where
  // there are both kinds, either wide items leave the single ones a share of the
  // CUs, at most a quarter, all in one round; or each kind has all CUs, which
  // costs a second round's start and end, some 6 us.  One round (measured against
  // two): 24 x 4 sequences over 5000 + 333 keys 24.5 us (28.9), 40 over 8000 + 100
  // 28 (40).  Two (against one): 64 over 16384 + 2048 152 us (244).
  const int w = p.launch.part[0].wide ? 0 : 1;
  int64_t cus_for[2] = {cus, cus};
  bool mixed = p.launch.part[0].wide != p.launch.part[1].wide && keys[0] > 0 && keys[1] > 0 && groups[1 - w] / 8 < cus / 2;
  if (mixed) {
    const double all = work[0] + work[1], share = work[w] < 0.75 * all ? 0.75 : work[w] / all;
    const double wide_us = work[w] / (share * (double)cus), narrow_us = work[1 - w] / ((1 - share) * (double)cus);
    mixed = (wide_us > narrow_us ? wide_us : narrow_us) < 6 + all / (double)cus;
    if (mixed) cus_for[w] = (int64_t)((double)cus * share);
  }
  p.mixed = mixed;
  for (int i = 0; i < 2; ++i) {
    const int s = i ? 1 - w : w;  // wide items first
    PartPlan &q = p.launch.part[s];
    if (keys[s] == 0) continue;
    const int64_t unit = a.kv.page > 64 ? a.kv.page : 64;  // a part of fewer keys costs more than reading them
    int64_t splits = (cus_for[s] * (q.wide ? 1 : 8) + (mixed ? groups[s] / 2 : 0)) / groups[s];
    if (q.wide && splits > 1 && splits * groups[s] > cus) --splits;
    // Two wavefronts a CU nearly fill the memory's bandwidth; more are for
    // chunks of 256 keys at least, as each costs a partial O.  One sequence of 8
    // heads x 4 over 16384 keys: 64 chunks 20 us, 256 24; 16 of them with 8000
    // keys each: 16 chunks 105 us, 4 121.
    if (!q.wide && !mixed) {
      const int64_t two = 2 * cus / groups[s], most = keys[s] / 256;
      if (splits > most) splits = most;
      if (splits < two) splits = two;
    }
    if (splits < 1) splits = 1;
    int64_t chunk = round_up((keys[s] + splits - 1) / splits, unit);
    const int64_t pages = q.wide ? WIDE_PAGES : NARROW_PAGES;
    const int64_t most = (pages - 1) * a.kv.page / unit * unit;
    if (chunk > most) chunk = most;
    q.splits = (int)((keys[s] + chunk - 1) / chunk);
    q.chunk = (int)(s ? unit : chunk);
    q.items = groups[s] * q.splits;
    if (mixed && q.wide && q.items < cus) cus_for[1 - s] = cus - q.items;
  }
  p.launch.part[1].part0 = p.launch.part[0].splits;
  p.parts = p.launch.part[0].splits + p.launch.part[1].splits;
  // one part alone writes the output: 64 sequences of up to 60 own keys 7.5 us (10.2
  // with a join), 256 of up to 512 54.5 (60.4),
  // 2048 tokens of 32 heads among themselves 68 (94)
  p.launch.direct = p.parts == 1;
  return p;
}

size_t attn_prefix_ws(const AttnArgs &a) {
  const Plan p = plan_for(a);
  return p.launch.direct ? 0 : (size_t)p.parts * (size_t)p.rows_all * ((size_t)a.kv.d * 4 + 8);
}

}  // namespace oq
