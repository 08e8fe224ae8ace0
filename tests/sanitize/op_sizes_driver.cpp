// Checks csrc/op_sizes.h, the sizes that the launchers of the bf16 / fp16 operators and their host code
// share, against counts made the long way round.
#include "op_sizes.h"

#include <cstdio>
#include <initializer_list>
#include <random>
#include <set>
#include <vector>

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

// Row counts of the groups as the kernels clamp them, and the rows behind them as one more.
static std::vector<int64_t> clamped(const std::vector<int64_t>& splits, int64_t M) {
  std::vector<int64_t> m;
  int64_t at = 0;
  for (int64_t s : splits) {
    const int64_t e = std::min(at + std::max<int64_t>(s, 0), M);
    m.push_back(e - at);
    at = e;
  }
  m.push_back(M - at);
  return m;
}
static int64_t tiles(const std::vector<int64_t>& m, size_t groups, int64_t h) {
  int64_t t = 0;
  for (size_t g = 0; g < groups; ++g) t += (m[g] + h - 1) / h;
  return t;
}

static void splits_of_every_kind(std::mt19937& r) {
  auto upto = [&](int64_t n) { return (int64_t)(r() % (uint64_t)(n + 1)); };
  for (int round = 0; round < 4000; ++round) {
    const int G = 1 + (int)upto(round % 3 ? 9 : 300);
    const int64_t M = round % 7 ? upto(3000) : upto(9);
    const int64_t n = 1 + upto(900), k = 1 + upto(900);
    std::vector<int64_t> s(G);
    const int kind = round % 5;
    for (int g = 0; g < G; ++g)
      s[g] = kind == 0 ? upto(2 * M / G) : kind == 1 ? 1 : kind == 2 ? (upto(9) ? 0 : upto(M)) : kind == 3 ? 128 * upto(3) + 1
                                                                                            : (int64_t)(int32_t)r();
    const std::vector<int64_t> m = clamped(s, M);
    for (int64_t h : {16, 32, 64, 128, 256}) {
      EXPECT(tiles(m, G, h) <= sizes::tiles_bound(M, G, h), "G %d M %lld h %lld", G, (long long)M, (long long)h);
      EXPECT(tiles(m, G + 1, h) <= sizes::row_tiles_bound(M, G, h), "G %d M %lld h %lld", G, (long long)M, (long long)h);
    }
    // the table's entries, and what its equal tile heights cover
    const int64_t words = (int64_t)(sizes::table_bytes(G, M) / 4) - sizes::kTableWords;
    EXPECT(std::max<int64_t>(tiles(m, G + 1, 256), G) * sizes::kTableWords <= words, "G %d M %lld", G, (long long)M);
    for (int64_t rows : m) {
      const int64_t nt = (rows + 255) / 256, h = nt ? ((rows + nt - 1) / nt + 31) / 32 * 32 : 0;
      EXPECT(h <= 256 && nt * h >= rows && (nt == 0 || (nt - 1) * h < rows), "rows %lld", (long long)rows);
    }
    // the ring kernel: every tile is some block's
    const int64_t ntn = (n + 127) / 128, total = tiles(m, G + 1, 128) * ntn, per = (total + 7) / 8;
    EXPECT(sizes::ring_blocks(false, G, M, n, k) >= 8 * per, "G %d M %lld n %lld", G, (long long)M, (long long)n);
    const int64_t tpg = ((n + 127) / 128) * ((k + 127) / 128), blocks = sizes::ring_blocks(true, G, M, n, k);
    std::set<std::pair<int64_t, int64_t>> seen;
    for (int64_t b = 0; b < blocks; ++b) {
      const int64_t eighth = (tpg + 7) / 8;
      const int64_t g = tpg >= 64 ? (b >> 3) / eighth : b / tpg, t = tpg >= 64 ? (b & 7) * eighth + (b >> 3) % eighth : b % tpg;
      if (t < tpg && g < G) EXPECT(seen.insert({g, t}).second, "tile twice: %lld %lld", (long long)g, (long long)t);
    }
    EXPECT((int64_t)seen.size() == G * tpg, "G %d n %lld k %lld", G, (long long)n, (long long)k);
    // parts: scratch for each, their stages together the contraction's
    for (bool w : {false, true}) {
      const int64_t parts = sizes::parts(w, G, M, n, k);
      EXPECT(parts >= 1 && parts <= 16, "%lld parts", (long long)parts);
      if (parts > 1) {
        EXPECT(parts * (w ? G * n * k : M * n) <= sizes::part_floats(w, G, M, n, k), "parts %lld", (long long)parts);
        const int64_t nst = ((w ? m[0] : k) + 63) / 64;
        int64_t at = 0;
        for (int64_t z = 0; z < parts; ++z) {
          EXPECT(nst * z / parts == at, "part %lld", (long long)z);
          at = nst * (z + 1) / parts;
        }
        EXPECT(at == nst, "parts %lld", (long long)parts);
      }
    }
    // chunks of the adapters' outer products
    const int64_t h = sizes::outer_rows(M, n);
    EXPECT(h % sizes::kOuterRows == 0 && h >= 256 && h <= 2048, "%lld", (long long)h);
    EXPECT(tiles(m, G, h) * 5 * n <= sizes::outer_part_floats(M, n, 5, G), "G %d M %lld", G, (long long)M);
  }
}

static void order() {
  for (int64_t n : {0, 1, 1023, 1024, 1025, 16384, 16385, 262144, 262145, 1000000, (1 << 30) - 1}) {
    const int64_t chunk = sizes::order_chunk(n), grid = sizes::order_grid(n);
    EXPECT(chunk % sizes::kOrderThreads == 0 && grid >= 1 && grid <= sizes::kOrderBlocks, "n %lld", (long long)n);
    EXPECT(grid * chunk >= n && (grid - 1) * chunk <= std::max<int64_t>(n - 1, 0), "n %lld", (long long)n);
    EXPECT(sizes::order_blocks(n) == (n > 16384 ? grid : 1), "n %lld", (long long)n);
  }
}

int main() {
  folded();
  std::mt19937 r(7);
  splits_of_every_kind(r);
  order();
  if (bad) return 1;
  printf("all sizes as counted\n");
  return 0;
}
