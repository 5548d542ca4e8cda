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
// (measured at K = 4096 in the table's order, with e8m0 scales: 299, 245, 192, 111, 67, 43, 30
// and 24 us; with fp16 scales 350, 290, 223, 131, 76, 50, 36 and 27 us).
constexpr Q4TileCost kQ4Tiles[] = {{256, 256, 1180}, {256, 192, 970}, {256, 128, 760},
                                   {128, 128, 440},  {64, 128, 270},  {64, 64, 185},
                                   {32, 64, 130},    {32, 32, 100}};

#if defined(__HIP__)
#define GEMM_F32_BOTH __host__ __device__
#else
#define GEMM_F32_BOTH
#endif

constexpr int kQ4Cus = 256;

// The groups that can have rows.
GEMM_F32_BOTH inline int q4_active(const Q4Problem& p) {
  return p.g.groups < p.g.rows ? p.g.groups : p.g.rows;
}

// Row tiles: one for each group that can have rows, and the last ones counted half full.
inline int64_t q4_row_tiles(const Q4Problem& p, int rows) {
  if (p.g.groups == 1) return ((int64_t)p.g.rows + rows - 1) / rows;
  const int64_t active = q4_active(p);
  return std::max(active, p.g.rows / rows + (active + 1) / 2);
}

inline int64_t q4_rounds(const Q4Problem& p, const Q4TileCost& t) {
  const int64_t tiles = q4_row_tiles(p, t.rows) * (((int64_t)p.g.N + t.cols - 1) / t.cols);
  return (tiles + kQ4Cus - 1) / kQ4Cus;
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

// Its waves along K, as a power of two: so many that a workgroup on each CU has columns
// for its waves, and no more than there are chunks.
GEMM_F32_BOTH inline int q4_waves_along_k(const Q4Problem& p) {
  const int64_t chunks = ((int64_t)p.g.K + kQ4FewK - 1) / kQ4FewK;
  const int64_t columns = ((int64_t)p.g.N + 15) / 16 * q4_active(p);
  int log2 = 0;
  while (log2 < kQ4FewWavesLog2 && (columns << log2) < (kQ4Cus << kQ4FewWavesLog2) &&
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

// Its strips of columns, one for the waves of a workgroup that do not share K.
GEMM_F32_BOTH inline int q4_few_strips(const Q4Problem& p) {
  const int wide = 16 << kQ4FewWavesLog2 >> q4_waves_along_k(p);
  return (int)(((int64_t)p.g.N + wide - 1) / wide);
}

// Whether the kernel for few rows (kernels_q4_few.hip) is the faster one.  In microseconds,
// with e strips of columns for each workgroup, row tiles of r rows, c chunks along K, of which
// a wave takes w for each strip, a round of the CUs takes
//   5 to 6 + 0.0215 r c (staging, for each strip where LDS has no room for all chunks)
//   + e (0.2 + 0.06 r + w (1.17 + 0.014 r))
// and tiles whose rounds cost t take 3 + t (3.9 + 4.3 K / 1024) / 100, and 4 where the waves
// of the smallest, which share K by 256, have a rest behind that.  These are fits over 275
// sizes, 1 to 128 groups of 1 to 48 rows each, 512 x 2048 to 8192 x 8192, e8m0 scales.  Over
// these and others with up to 200 rows a group the choices by them take 1.4 % longer than the
// faster kernel on average, and 4 % where groups have from half to three halves of the
// average.  (Groups are counted as even, the largest with one row more: the offsets that say
// better are the device's.  Few against tiles in us.
// 4096 x 4096: 8 rows 15 against 23, 24 rows 30 against 24; 8192 x 8192: 8 rows 26 against 38;
// 32 groups of 2048 x 1024: 8 rows each 17 against 45, 32 rows 34 against 45, 48 rows 52
// against 47; of 7168 x 2048: 8 rows each 86 against 236, 32 rows 214 against 251, 48 rows
// 384 against 255.)
inline bool q4_few(const Q4Problem& p) {
  if (p.g.K < kQ4FewK) return false;
  const bool one = p.g.groups == 1;
  const int most = q4_few_rows(p), active = q4_active(p);
  const bool small = !one && p.g.rows <= (int64_t)active * most;   // a tile each
  const double tiles = small ? active : (double)q4_row_tiles(p, most);
  const double strips = q4_few_strips(p), chunks = (p.g.K + kQ4FewK - 1) / kQ4FewK;
  const double w = std::ceil(chunks / (1 << q4_waves_along_k(p)));
  const double r = one ? std::ceil(p.g.rows / tiles)
                       : std::min((double)most, (double)p.g.rows / active + 1);
  const double e = std::ceil(strips / std::max(1.0, std::floor(kQ4Cus / tiles)));
  const double rounds = std::ceil(tiles / kQ4Cus);
  const double fixed = !one ? 5.5 : tiles > 1 ? 6 : 5;
  const double staged = 0.0215 * r * chunks * (chunks * r > 200 ? e : 1.0);
  const double few = rounds * (fixed + staged + e * (0.2 + 0.06 * r + w * (1.17 + 0.014 * r)));
  const Q4Tile t = q4_tile(p);
  const double rest = t == kTile32 && p.g.K > 256 && p.g.K % 256 != 0 ? 4 : 0;
  return few < 3 + rest + 1e-2 * (double)q4_tile_cost(p, t) * (3.9 + 4.3 / 1024 * p.g.K);
}

}  // namespace gemmf32
