// Which kernel a product with 4-bit weights takes: rules on sizes alone.  Host code
// without a HIP call.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "experts_internal.h"

namespace gemmf32 {

enum Q4Tile {
  kTile256, kTile256x192, kTile256x128, kTile128, kTile64x128, kTile64, kTile32x64, kTile32
};

struct Q4TileCost {
  int rows, cols;
  int round;   // time of a round of the CUs, one workgroup on each, that of kTile32 being 100
};

// A CU holds one workgroup of each tile, so a product takes as long as the rounds its
// workgroups make, times the round's time, which grows with K alike for all of them
// (measured at K = 4096 in the table's order, with e8m0 scales: 292, 238, 189, 107, 70, 47, 33
// and 26 us; with fp16 scales 343, 284, 220, 130, 75, 51, 38 and 28 us).
constexpr Q4TileCost kQ4Tiles[] = {{256, 256, 1180}, {256, 192, 970}, {256, 128, 760},
                                   {128, 128, 440},  {64, 128, 270},  {64, 64, 185},
                                   {32, 64, 130},    {32, 32, 100}};

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

constexpr int kQ4FewK = 128;   // the least K that the kernel for few rows takes, and its chunk
constexpr int kQ4FewWavesLog2 = 4;
constexpr int kQ4FewRows = 20, kQ4FewRowsDeep = 12;

#if defined(__HIP__)
#define GEMM_F32_BOTH __host__ __device__
#else
#define GEMM_F32_BOTH
#endif

// Its waves along K, as a power of two: so many that a workgroup on each CU has columns
// for its waves, and no more than there are chunks.
GEMM_F32_BOTH inline int q4_waves_along_k(const Q4Problem& p) {
  const int64_t chunks = ((int64_t)p.g.K + kQ4FewK - 1) / kQ4FewK;
  const int64_t columns = ((int64_t)p.g.N + 15) / 16 * p.g.groups;
  int log2 = 0;
  while (log2 < kQ4FewWavesLog2 && (columns << log2) < (256 << kQ4FewWavesLog2) &&
         (INT64_C(1) << log2) < chunks)
    ++log2;
  return log2;
}

// Rows of its row tiles, at most: those whose parts of a chunk for each wave along K fit
// into LDS, of two chunks where K takes several passes over 8 waves (8192 x 8192, 16 rows:
// 47 us with one).
GEMM_F32_BOTH inline int q4_few_rows(const Q4Problem& p) {
  const int log2 = q4_waves_along_k(p);
  const bool deep = log2 == kQ4FewWavesLog2 ||
                    (log2 == kQ4FewWavesLog2 - 1 && p.g.K > kQ4FewK << log2);
  return deep ? kQ4FewRowsDeep : kQ4FewRows;
}

// Whether the kernel for few rows (kernels_q4_few.hip) is the faster one, by its time in
// the tiles' unit: with e strips of columns for each workgroup, c columns of 16 in them,
// and r rows a row tile takes 12 + 2 r + c (9 + 0.8 r), and 14 for each strip where all
// waves go along K.  Row tiles of one matrix go beside each other, those of a group one
// after another; uneven groups are counted half as long again as their average.
// (Few against tiles in us, e8m0 scales.  4096 x 4096: 8 rows 15 against 23, 12 rows 18
// against 23, 16 rows 24 against 23; 8192 x 8192: 8 rows 25 against 39, 12 rows 32 against
// 39, 16 rows 42 against 39; 28672 x 8192: 16 rows 97 against 97, 24 rows 148 against 96;
// 2048 x 1024 in 32 groups: 6 rows each 17 against 47, 32 rows 42 against 48.)
inline bool q4_few(const Q4Problem& p) {
  if (p.g.K < kQ4FewK) return false;
  const int waves = 1 << kQ4FewWavesLog2, wide = waves >> q4_waves_along_k(p);
  const auto up = [](double x, double by) { return std::ceil(x / by); };
  const bool one = p.g.groups == 1;
  const double strips = up(p.g.N, 16 * wide), groups = p.g.groups;
  const double rows = one ? p.g.rows : 1.5 * p.g.rows / groups + 1;
  const double tiles = up(rows, q4_few_rows(p)), r = up(rows, tiles);
  const double beside = groups * (one ? tiles : 1.0), turns = one ? 1.0 : tiles;
  const double e = up(strips, std::max(1.0, std::floor(256 / beside)));
  const double rounds = up(beside * up(strips, e), 256);
  const double time =
      12 + 2 * r + e * wide * (9 + 0.8 * r) + (wide == 1 ? 14 * e : 0.0);
  return time * rounds * turns < 0.88 * (double)q4_tile_cost(p, q4_tile(p));
}

}  // namespace gemmf32
