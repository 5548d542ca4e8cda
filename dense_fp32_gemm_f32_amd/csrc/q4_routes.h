// Which kernel a product with 4-bit weights takes: rules on sizes alone.  Host code
// without a HIP call.
#pragma once

#include <algorithm>
#include <cstdint>

#include "experts_internal.h"

namespace gemmf32 {

enum Q4Tile { kTile256, kTile128, kTile64x128, kTile64, kTile32x64, kTile32 };

struct Q4TileCost {
  int rows, cols;
  int round;   // time of a round of the CUs, one workgroup on each, that of kTile32 being 100
};

// A CU holds one workgroup of each tile, so a product takes as long as the rounds its
// workgroups make, times the round's time, which grows with K alike for all of them
// (measured at K = 4096 with e8m0 scales: 24, 31, 45, 68, 104 and 275 us; with fp16 scales
// 27, 37, 53, 78, 126 and 333 us).
constexpr Q4TileCost kQ4Tiles[] = {{256, 256, 1150}, {128, 128, 435}, {64, 128, 285},
                                   {64, 64, 190},    {32, 64, 132},   {32, 32, 100}};

// Rounds of a tile: the groups' last row tiles are counted half full.
inline int64_t q4_rounds(const Q4Problem& p, const Q4TileCost& t) {
  const int64_t row_tiles = p.g.groups == 1
                                ? ((int64_t)p.g.rows + t.rows - 1) / t.rows
                                : (int64_t)p.g.rows / t.rows +
                                      (std::min(p.g.groups, p.g.rows) + 1) / 2;
  return (row_tiles * (((int64_t)p.g.N + t.cols - 1) / t.cols) + 255) / 256;
}

inline int64_t q4_tile_cost(const Q4Problem& p, int t) {
  return q4_rounds(p, kQ4Tiles[t]) * kQ4Tiles[t].round;
}

inline Q4Tile q4_tile(const Q4Problem& p) {
  int best = kTile32;
  for (int t = kTile32 - 1; t >= 0; --t)
    if (q4_tile_cost(p, t) < q4_tile_cost(p, best)) best = t;
  return (Q4Tile)best;
}

// The kernel for few rows (kernels_q4_few.hip), whose row tiles have up to 8, in the same
// unit: with c columns of 16 for each CU, a row tile takes as long as (0.3 + 0.12 c)
// rounds of kTile32; where columns are fewer than CUs, row tiles go beside each other.
// (e8m0 scales, 4096 x 4096: 8 rows 14 us against 24 us for the tiles, 16 rows 23 against
// 24, 24 rows 39 against 24; 8192 x 8192: 8 rows 25 against 40, 16 rows 44 against 40;
// 2048 x 1024 in 32 groups: 192 rows 17 against 48, 700 rows 42 against 51, 1000 rows 54
// against 53.)
inline int64_t q4_few_cost(const Q4Problem& p) {
  const int64_t columns = ((int64_t)p.g.N + 15) / 16 * p.g.groups;   // 256 to a round
  // row tiles of a group, in quarters; of uneven groups a little more than their average
  const int64_t tiles = p.g.groups == 1
                            ? ((int64_t)p.g.rows + 7) / 8 * 4
                            : std::max((int64_t)4, (int64_t)p.g.rows / (2 * p.g.groups) + 1);
  if (columns < 256) return 30 + 25 * columns * tiles / (4 * 256);
  return tiles * (30 + 12 * columns / 256) / 4;
}

constexpr int kQ4FewK = 128;   // the least K it takes

inline bool q4_few(const Q4Problem& p) {
  return p.g.K >= kQ4FewK && q4_few_cost(p) < q4_tile_cost(p, q4_tile(p));
}

}  // namespace gemmf32
