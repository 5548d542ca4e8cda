// Grouped products with few rows in a group, or few columns (gfx950): a workgroup
// owns 16 or 32 places of one group by 16 NB columns, K split over its waves
// (grouped_rows.h).
#include "grouped_rows.h"

namespace gemmf32 {
namespace {

using namespace grouped;

template <int kWaves, int RM, int NB, bool kTB, int U, bool kOnce>
__device__ __forceinline__ void rows_tile(float* red, const GroupedProblem& p, const Epilogue& ep,
                                          int g, int m0, int end, int n0, int wave, int lane) {
  rows_product<kWaves, RM, NB, kTB, U, kOnce>(
      red, p.A, p.lda,
      [&](int i) {
        if (m0 + i >= end) return -1;
        const int r = p.ia ? p.ia[m0 + i] : m0 + i;
        return r >= 0 && r < p.rows_a ? r : -1;
      },
      p.B + g * p.sb, p.ldb, p.N, n0, p.K, wave, lane);
  constexpr int BM = 16 * RM, BN = 16 * NB;
  const float scale = p.gscale ? p.gscale[g] : 1.f;
  Epilogue e = ep;
  if (e.bias) e.bias += g * p.sbias;
  for (int x = threadIdx.x; x < BM * BN; x += kWaves * 64) {
    const int at = m0 + x / BN, col = n0 + x % BN;
    if (at >= end || col >= p.N) continue;
    const int r = p.ic ? p.ic[at] : at;
    if (r < 0 || r >= p.rows_c) continue;
    float* out = p.C + (int64_t)r * p.ldc + col;
    *out = epilogue_apply(e, scale * rows_sum<kWaves, RM, NB>(red, x), out, col);
  }
}

template <int kWaves, int RM, int NB, bool kTB, int U, bool kOnce>
__global__ void __launch_bounds__(kWaves * 64)
    grouped_rows_kernel(GroupedProblem p, Epilogue ep, int strips, unsigned cap) {
  constexpr int BM = 16 * RM;
  __shared__ float red[kWaves * BM * 16 * NB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  RowTiles rt{p.offsets, p.groups, p.rows, BM, lane, cap, 0};
  const unsigned total = rt.total();
  // each XCD takes a contiguous range of the tiles, strips of a group together
  const int id = xcd_position(tile_id(), total * (unsigned)strips);
  if (id < 0) return;
  const unsigned t = (unsigned)id / strips;
  int g = 0, begin = 0, end = 0;
  unsigned first = 0;
  if (!rt.find(t, g, begin, end, first)) return;
  const int m0 = begin + (int)(t - first) * BM, n0 = (int)(id % strips) * 16 * NB;
  if (RM == 1 || end - m0 <= 16) {
    rows_tile<kWaves, 1, NB, kTB, U, kOnce>(red, p, ep, g, m0, min(end, m0 + 16), n0, wave, lane);
  } else {
    rows_tile<kWaves, RM, NB, kTB, U, kOnce>(red, p, ep, g, m0, min(end, m0 + BM), n0, wave, lane);
  }
}

// kWaves waves, chunks of 16 kU k; with B stored K x N and 16 places a strip's runs of
// whole lines are read once and non-temporally (64 groups of 1024 x 1024, weights not
// in a cache: 51 against 56 us; stored N x K a load reads half lines, which a
// non-temporal load fetches twice: 56 against 54 us).  Not with 32 places, whose
// groups may have several tiles (13 groups of 161, 769 x 1001: 61 against 70 us; 64 of
// 24, 1024 x 1024: 66 against 69).
template <int kWaves, int RM, int NB, bool kTB, int kU>
hipError_t launch(const GroupedProblem& p, const Epilogue& e, hipStream_t s) {
  const int64_t strips = ((int64_t)p.N + 16 * NB - 1) / (16 * NB);
  const int64_t cap = most_row_tiles(p.rows, p.groups, 16 * RM);
  if (cap * strips > 0x7fffffff) return hipErrorInvalidConfiguration;
  constexpr bool kOnce = !kTB && RM == 1 && (kWaves == 4 || (kWaves == 16 && NB == 2));
  hipLaunchKernelGGL((grouped_rows_kernel<kWaves, RM, NB, kTB, kU, kOnce>), tile_grid(cap * strips),
                     dim3(kWaves * 64), 0, s, p, e, (int)strips, (unsigned)cap);
  return hipGetLastError();
}

// Many workgroups: 64 columns each, in 4 waves that look one step ahead, so that
// four workgroups share a CU (B stored K x N, 32 x 1024 x 2048 with 6 places a group:
// 49 us against 52 us for 8 waves that look two steps ahead; stored N x K, 64 groups
// of 24, 1024 x 1024: 58 against 72 us for 8 waves of chunks of 64 k); with 16 places
// and B stored N x K those 8 waves (64 groups of one, 1024 x 2048: 97 against 111 us).
template <int RM>
hipError_t launch_many(const GroupedProblem& p, const Epilogue& e, hipStream_t s) {
  if (!p.tb) return launch<4, RM, 4, false, 1>(p, e, s);
  if constexpr (RM == 1)
    return launch<8, 1, 4, true, 4>(p, e, s);
  else
    return launch<4, RM, 4, true, 1>(p, e, s);
}

// Few workgroups: 16 waves each, 32 or 16 columns.
template <int RM, bool kTB>
hipError_t launch_few(const GroupedProblem& p, int nb, const Epilogue& e, hipStream_t s) {
  return nb == 1 ? launch<16, RM, 1, kTB, 1>(p, e, s) : launch<16, RM, 2, kTB, 1>(p, e, s);
}

// Few columns: 16 places a workgroup, 8 waves, all columns in one strip.
template <bool kTB>
hipError_t launch_thin(const GroupedProblem& p, const Epilogue& e, hipStream_t s) {
  if (p.N <= 16) return launch<8, 1, 1, kTB, 4>(p, e, s);
  if (p.N <= 32) return launch<8, 1, 2, kTB, 4>(p, e, s);
  return launch<8, 1, 4, kTB, kTB ? 4 : 2>(p, e, s);
}

}  // namespace

hipError_t launch_grouped_rows(const GroupedProblem& p, const Epilogue& e, hipStream_t s) {
  // few columns (4096 places of 2048, 32 columns: 14 us against 20 us for 32 places
  // a workgroup)
  if (p.N <= 64) return p.tb ? launch_thin<true>(p, e, s) : launch_thin<false>(p, e, s);
  // few rows in a group: 32 places a workgroup where groups have more than 10 on
  // average (16 groups of 19, 1024 x 1024: 19 against 24 us), else 16 (less LDS: 6
  // places, 32 x 1024 x 2048: 47 against 51 us)
  const int64_t busy = p.rows < p.groups ? p.rows : p.groups;
  const bool two = p.rows > 10 * busy;
  const int64_t tiles = busy * ((p.rows / busy + (two ? 31 : 15)) / (two ? 32 : 16));
  // strips of 64 columns where they leave two workgroups a CU, of 32 where those
  // leave one (8 groups of one place, 2048 x 1024: 15 us against 22 and 18 us for 64
  // and 16 columns; one of 4096 x 4096: 16 us for 16 columns against 21 for 32)
  if (tiles * (((int64_t)p.N + 63) / 64) >= 512)
    return two ? launch_many<2>(p, e, s) : launch_many<1>(p, e, s);
  const int nb = tiles * (((int64_t)p.N + 31) / 32) >= 256 ? 2 : 1;
  if (p.tb) return two ? launch_few<2, true>(p, nb, e, s) : launch_few<1, true>(p, nb, e, s);
  return two ? launch_few<2, false>(p, nb, e, s) : launch_few<1, false>(p, nb, e, s);
}

}  // namespace gemmf32
