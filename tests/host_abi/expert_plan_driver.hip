// The plan of the experts' products on the CPU.  Arguments: any number of groups
// of "n K N E act"; prints for each "mt ks columns grid".  Without arguments it
// checks the plan over the ranges of its sizes and prints "<n> cases passed".
#include <cstdio>
#include <cstdlib>

#include "serve_stubs.h"
#include "sparse_plan.h"

namespace {

int g_cases = 0, g_fail = 0;

void truth(bool ok, long long n, int K, int N, int E, int act) {
  ++g_cases;
  if (!ok && ++g_fail < 50) std::printf("n %lld K %d N %d E %d act %d: wrong\n", n, K, N, E, act);
}

// Row tiles of n entries: spread evenly (0), one for every expert and the rest for the last
// (1), or one more than a tile for as many as there are (2).
int64_t row_tiles(int64_t n, int E, int rows, int how) {
  int64_t tiles = 0, left = n;
  for (int e = 0; e < E; ++e) {
    const int64_t want = how == 0 ? n / E + (e < n % E) : how == 1 ? 1 : rows + 1, c = e == E - 1 || want > left ? left : want;
    tiles += (c + rows - 1) / rows;
    left -= c;
  }
  return tiles;
}

void ranges() {
  for (int cus : {1, 64, 256, 304}) {
    g_cus = cus;
    for (int act = 0; act < 2; ++act)
      for (int64_t n : {1ll, 2ll, 15ll, 16ll, 17ll, 100ll, 1023ll, 4096ll, 33000ll, 524288ll, 1ll << 28})
        for (int E : {1, 2, 8, 60, 64, 65, 128, 1000, 1024})
          for (int N : {2, 34, 256, 258, 1536, 4096, 65536, 1 << 20})
            for (int K : {16, 128, 384, 400, 4096, 131056}) {
              const oq::ExpertPlan p = oq::expert_plan(n, K, N, E, act);
              const int rows = p.mt ? 16 * p.mt : oq::EXPERT_BM, wide = p.mt ? 256 / p.ks : oq::EXPERT_BN;
              bool ok = (p.mt == 0 && p.ks == 1) || (p.mt == 4 && p.ks == 1) || (p.mt == 1 && (p.ks == 1 || p.ks == 2 || p.ks == 4 || p.ks == 8));
              ok = ok && (p.mt || K > 128 * (oq::EXPERT_STAGES - 1));
              ok = ok && p.columns * wide >= N && (p.columns - 1) * wide < N && p.grid % 8 == 0;
              // whatever the lists are, no tile is without a workgroup
              for (int how = 0; how < 3; ++how) ok = ok && row_tiles(n, E, rows, how) * p.columns <= p.grid;
              // outputs that fit a GPU's memory (2^38 bytes) never need more workgroups than the kernels count
              if ((double)n * (act ? N / 2 : N) * 2 <= 274877906944.) ok = ok && p.grid <= 0x7fffffff;
              truth(ok, n, K, N, E, act);
            }
  }
  g_cus = 256;
  // a launch's workgroups stay below 2^32 threads
  for (int64_t threads : {64ll, 256ll, 512ll, 1024ll, 262144ll}) {
    const int64_t rows = oq::rows_of_launch(threads);
    truth(rows >= 1 && rows * threads < 1ll << 32 && (rows + 1) * threads >= 1ll << 32, threads, 0, 0, 0, 0);
  }
}

}  // namespace

int main(int argc, char **argv) {
  if (argc == 1) {
    ranges();
    if (g_fail) return 1;
    std::printf("%d cases passed\n", g_cases);
    return 0;
  }
  for (int i = 1; i + 4 < argc; i += 5) {
    const oq::ExpertPlan p = oq::expert_plan(std::atoll(argv[i]), std::atoi(argv[i + 1]), std::atoi(argv[i + 2]), std::atoi(argv[i + 3]), std::atoi(argv[i + 4]));
    std::printf("%d %d %lld %lld\n", p.mt, p.ks, (long long)p.columns, (long long)p.grid);
  }
  return 0;
}
