// Launch and scratch sizes of the operators around the experts (routing, norms, 4-bit products), shared by
// their launchers and their host code.  Plain C++.
#pragma once
#include "op_sizes.h"

namespace gmlp {
namespace sizes {

// ----------------------------------------------------------------------------- norms
// Threads of a row in eights of C a thread, whole waves.
inline int norm_threads(int64_t H, int C) { return (int)(((H + 7) / 8 + 64 * C - 1) / (64 * C) * 64); }
// Workgroups of the backward, and so the parts that its column sums have: what fills the device with waves of eights,
// but four rows a workgroup where that leaves one on a CU (each writes its sums, which are read once more).
constexpr int kNormCus = 256;
inline int norm_bwd_blocks(int64_t T, int64_t H) {
  const int64_t per = std::min<int64_t>(std::max<int64_t>(1024 / norm_threads(H, 1), 1), 4);
  return (int)std::max<int64_t>(std::min<int64_t>(std::max<int64_t>(T / 4, kNormCus), std::min<int64_t>(T, kNormCus * per)), 1);
}
// Up to three column sums (weight, branch_weight, a gate by channel) of H columns a part.
inline int64_t norm_part_floats(int64_t T, int64_t H) { return 3 * (int64_t)norm_bwd_blocks(T, H) * H; }

// ----------------------------------------------------------------------------- products with 4-bit weights
constexpr int kW4Chunk = 128;        // elements along K that a wave takes at once
// Waves that share a tile's chunks where the tiles alone leave the device empty.
inline int w4_waves(int64_t K) { return (int)std::min<int64_t>(8, (K + kW4Chunk - 1) / kW4Chunk); }
// Workgroups with the smallest tile, 16 rows x 16 columns: what every launch stays below.
inline int64_t w4_tiles_bound(int64_t M, int64_t G, int64_t N) { return row_tiles_bound(M, (int)G, 16) * ((N + 15) / 16); }

}  // namespace sizes
}  // namespace gmlp
