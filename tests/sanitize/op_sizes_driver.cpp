// Checks csrc/op_sizes.h, the sizes that the launchers of the bf16 / fp16 operators and their host code
// share, against counts made the long way round.
#include "op_sizes.h"

#include <cstdio>
#include <initializer_list>

using namespace gmlp;

static int bad = 0;
#define EXPECT(c, ...) do { if (!(c)) { printf("%s: ", #c); printf(__VA_ARGS__); printf("\n"); ++bad; } } while (0)

// Every launch that fits one is one; the others cover their blocks with less than 2^32 threads along x, whole
// rounds over the XCDs, less than a row of blocks too many and no more rows than HIP takes.
static void folded() {
  for (int threads : {64, 256, 512, 1024})
    for (int sh = 0; sh <= 36; ++sh)
      for (int64_t d = -9; d <= 9; ++d) {
        const int64_t blocks = (int64_t(1) << sh) + d;
        if (blocks < 1) continue;
        const FoldedGrid g = fold_grid(blocks, threads);
        EXPECT((int64_t)g.x * threads < (int64_t(1) << 32), "%lld x %d", (long long)blocks, threads);
        EXPECT((int64_t)g.x * g.y >= blocks && (int64_t)g.x * (g.y - 1) < blocks, "%lld x %d", (long long)blocks, threads);
        EXPECT(g.y <= 65535, "%lld x %d", (long long)blocks, threads);
        EXPECT(g.y == 1 || g.x % 8 == 0, "%lld x %d", (long long)blocks, threads);
        EXPECT(g.y == 1 || blocks * threads >= (int64_t(1) << 32) - 8 * threads, "%lld x %d", (long long)blocks, threads);
      }
}

int main() {
  folded();
  if (bad) return 1;
  printf("all sizes as counted\n");
  return 0;
}
