// Sizes that the host code of the 16-bit operators computes: launches, tiles and scratch.  Plain C++.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

namespace gmlp {

// A launch of `blocks` workgroups.  A launch's threads along x are counted in 32 bits (2^24 + 5 workgroups of
// 256 ran as 5, without an error), so more workgroups than that are folded over y: the kernel's block
// number is blockIdx.x + blockIdx.y x, and numbers from `blocks` on have nothing to do.  x is an argument of
// the kernels: gridDim would add 256 bytes to what every launch writes for them.
struct FoldedGrid {
  uint32_t x, y;
};
inline FoldedGrid fold_grid(int64_t blocks, int threads) {
  const int64_t most = ((int64_t(1) << 32) - 1) / threads / 8 * 8;      // whole rounds over the eight XCDs
  if (blocks <= most) return {(uint32_t)blocks, 1};
  return {(uint32_t)most, (uint32_t)((blocks + most - 1) / most)};
}

namespace sizes {

// ----------------------------------------------------------------------------- tiles
// The most tiles of h rows that M rows in `groups` groups of any sizes give: each group has less than one
// tile of padding.
inline int64_t tiles_bound(int64_t M, int64_t groups, int64_t h) { return (M + (h - 1) * std::min<int64_t>(groups, M)) / h; }

// ----------------------------------------------------------------------------- group order
constexpr int kOrderThreads = 1024;
constexpr int kOrderBlocks = 256;
// Up to here every block counts all slots by itself, past it a pass of its own does.  Measured (us in a
// graph, own pass / by itself): 64 groups: 2048 slots 6.0 / 4.6, 6144 6.2 / 5.2, 16384 6.3 / 6.0, 24576
// 6.5 / 6.8, 65536 6.5 / 10.7; 1024 groups: 2048 slots 8.5 / 7.5, 16384 10.2 / 8.9, 65536 14.5 / 13.6.
constexpr int64_t kOrderAlone = 16384;
inline int64_t order_chunk(int64_t n) {           // slots of a block, whole rounds of its threads
  const int64_t per = (n + kOrderBlocks - 1) / kOrderBlocks;
  return std::max<int64_t>((per + kOrderThreads - 1) / kOrderThreads, 1) * kOrderThreads;
}
inline int order_grid(int64_t n) { return (int)std::max<int64_t>((n + order_chunk(n) - 1) / order_chunk(n), 1); }
inline int order_blocks(int64_t n) { return n > kOrderAlone ? order_grid(n) : 1; }      // of the counting pass

// ----------------------------------------------------------------------------- grouped products
constexpr int kTableWords = 8;                    // of a row tile's entry, behind as many for the count
// Row tiles of height h when the M rows are spread evenly.
inline int64_t row_tiles_even(int64_t M, int G, int h) {
  const int64_t used = std::min<int64_t>(G, std::max<int64_t>(M, 1));
  return used * ((M / used + h - 1) / h);
}
// Row tiles of the groups and, as one more, of the rows behind them.
inline int64_t row_tiles_bound(int64_t M, int G, int h) { return tiles_bound(M, (int64_t)G + 1, h); }
// The stream kernel's table: an entry per row tile of 256 (wgrad: per group).
inline size_t table_bytes(int G, int64_t M) {
  return 4 * (kTableWords + (size_t)std::max<int64_t>(row_tiles_bound(M, G, 256), G) * kTableWords);
}
// Workgroups of the ring kernel, tiles of 128 x 128: whole eighths for the XCDs.
inline int64_t ring_blocks(bool wgrad, int G, int64_t M, int64_t n, int64_t k) {
  const int64_t tn = (n + 127) / 128, tk = (k + 127) / 128, tpg = tn * tk;
  const int64_t grid = !wgrad ? 8 * ((row_tiles_bound(M, G, 128) * tn + 7) / 8) : tpg >= 64 ? 8 * ((tpg + 7) / 8) * G : tpg * G;
  return std::max<int64_t>(grid, 8);
}
// Parts of the contraction: with fewer tiles than CUs and eight stages or more, as many as fill the
// device twice, none shorter than four stages (one part where there is no tile at all).
inline int parts(bool wgrad, int G, int64_t M, int64_t n, int64_t k) {
  const int64_t tn = (n + 127) / 128, tk = (k + 127) / 128;
  const int64_t tiles = wgrad ? G * tn * tk : row_tiles_even(M, G, 128) * tn;
  const int64_t stages = ((wgrad ? M / std::min<int64_t>(G, std::max<int64_t>(M, 1)) : k) + 63) / 64;
  if (tiles == 0 || tiles >= 256 || stages < 8) return 1;
  return (int)std::max<int64_t>(1, std::min<int64_t>({512 / tiles, stages / 4, 16}));
}
inline int64_t part_stride(bool wgrad, int G, int64_t M, int64_t n, int64_t k) { return wgrad ? G * n * k : M * n; }
inline int64_t part_floats(bool wgrad, int G, int64_t M, int64_t n, int64_t k) {
  const int p = parts(wgrad, G, M, n, k);
  return p > 1 ? p * part_stride(wgrad, G, M, n, k) : 0;
}

// ----------------------------------------------------------------------------- adapters' outer products
constexpr int kOuterRows = 64, kOuterCols = 256;  // a stage's positions, a workgroup's columns
// Positions of a chunk: about 512 workgroups over the tensor, at least 256 (the chunks' results are
// written and read once more) and at most 2048.  Measured (bf16, us, db alone, chunks of 256, 512, 1024, 2048):
//   4096 rows x 4096   rank 16  20.4 26.0 26.1 26.1   rank 64  52.2 47.0 46.6 47.0    taken: 256
//  16384 rows x 4096            46.3 36.7 46.0 74.6             107 87.4  128  122           512
//  32768 rows x 4096            73.2 70.7 62.1 87.1             204  163  141  234          1024
//  16384 rows x 1024            20.5 25.7 41.2 73.2            30.9 40.3 64.2  114           256
//  32768 rows x 2048            43.2 36.8 47.2 74.8            97.0 80.1 72.0  118           512
inline int outer_rows(int64_t M, int64_t C) {
  const int64_t r = M * ((C + kOuterCols - 1) / kOuterCols) / 512;
  return (int)(std::min<int64_t>(std::max<int64_t>(r, 256), 2048) + kOuterRows - 1) / kOuterRows * kOuterRows;
}
inline int64_t outer_part_floats(int64_t M, int64_t C, int R, int L) { return tiles_bound(M, L, outer_rows(M, C)) * R * C; }

}  // namespace sizes
}  // namespace gmlp
