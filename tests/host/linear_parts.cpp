// Every launch's parts of K against the workspace that the entry points ask
// for, over sizes of all the rules' branches.
#include <cstdio>
#include <cstdlib>

#include "linear_plan.hpp"

using namespace muon;

static long cases = 0, cut = 0;

static void fits(const char *what, int32_t splits, int64_t rows, int64_t N, size_t have, int64_t M, int64_t K, int32_t groups) {
  ++cases;
  if (splits < 1 || splits > 32) std::printf("%s: %d parts\n", what, splits), std::exit(1);
  if (splits == 1) return;
  ++cut;
  const size_t need = (size_t)splits * (size_t)rows * (size_t)N * 4;
  if (need > have) {
    std::printf("%s: %ld x %ld x %ld, %d groups: %zu bytes for %zu\n", what, (long)M, (long)N, (long)K, groups, have, need);
    std::exit(1);
  }
}

int main() {
  const int64_t rows[] = {1, 2, 3, 4, 5, 7, 8, 9, 16, 63, 64, 65, 100, 128, 500, 1021, 2048, 4091, 32768, 131072};
  const int64_t sizes[] = {1, 3, 8, 40, 64, 128, 250, 256, 257, 512, 1000, 1024, 2047, 2048, 4096, 4104, 8192, 11008, 16384, 16392, 32768, 65536, 262144};
  const int32_t groups[] = {1, 2, 3, 7, 8, 32, 64, 256, 1024};
  for (int64_t M : rows)
    for (int64_t N : sizes)
      for (int64_t K : sizes)
        for (int32_t g : groups) {
          const size_t forward = linear_partial_bytes(M, N, K, g, false);
          for (int bf16 = 0; bf16 < 2; ++bf16) {
            fits("product", linear_plan(M, N, K, g, false, bf16).splits, M, N, forward, M, K, g);
            for (int bx = 0; bx < 2; ++bx)
              for (int grouped = g > 1; grouped < 2; ++grouped)
                if (few_rows(M, bf16, bx, grouped)) {
                  const FewPlan p = few_plan(M, N, K, g, bf16, bx);
                  fits("few rows", p.splits, M, N, forward, M, K, g);
                  if (p.tiles_m < 1 || p.tiles_m > FEW_ROWS || (int64_t)p.tiles_n * (bx ? FEW_ACROSS : FEW_ADJACENT) < N) return 1;
                }
            // a gradient's M and N are the weights' sides, its K the rows
            fits("weights' gradient", linear_plan(N, K, M, g, true, bf16).splits, N * g, K, linear_partial_bytes(N, K, M, g, true), N, M, g);
          }
        }
  std::printf("linear parts ok: %ld launches, %ld in parts\n", cases, cut);
  return 0;
}
