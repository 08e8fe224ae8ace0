// Sizes that the host code of the 16-bit operators computes: launches, tiles and scratch.  Plain C++.
#pragma once
#include <stdint.h>

namespace gmlp {

// A launch of `blocks` workgroups.  A launch's threads along x are counted in 32 bits (2^24 + 5 workgroups of
// 256 ran as 5, without an error), so more workgroups than that are folded over y: the kernel's block
// number is x + y gridDim.x, and numbers from `blocks` on have nothing to do.
struct FoldedGrid {
  uint32_t x, y;
};
inline FoldedGrid fold_grid(int64_t blocks, int threads) {
  const int64_t most = ((int64_t(1) << 32) - 1) / threads / 8 * 8;      // whole rounds over the eight XCDs
  if (blocks <= most) return {(uint32_t)blocks, 1};
  return {(uint32_t)most, (uint32_t)((blocks + most - 1) / most)};
}

}  // namespace gmlp
