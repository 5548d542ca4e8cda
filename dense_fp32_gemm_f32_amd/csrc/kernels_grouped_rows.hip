// Grouped products with few rows in a group, or few columns (gfx950): a workgroup
// owns 16 or 32 places of one group by 16 NB columns, K split over its waves
// (grouped_rows.h).
#include "grouped_rows.h"

namespace gemmf32 {
namespace {

using namespace grouped;

template <int RM, int NB, bool kTB, int U>
__device__ __forceinline__ void rows_tile(float* red, const GroupedProblem& p, const Epilogue& ep,
                                          int g, int m0, int end, int n0, int wave, int lane) {
  rows_product<RM, NB, kTB, U>(
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
    *out = epilogue_apply(e, scale * rows_sum<RM, NB>(red, x), out, col);
  }
}

template <int NB, bool kTB, int U>
__global__ void __launch_bounds__(kWaves * 64)
    grouped_rows_kernel(GroupedProblem p, Epilogue ep, int strips, unsigned cap) {
  __shared__ float red[kWaves * 32 * 16 * NB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  RowTiles rt{p.offsets, p.groups, p.rows, 32, lane, cap, 0};
  const unsigned total = rt.total();
  const unsigned id = tile_id(), t = id / strips;
  if (t >= total) return;
  int g = 0, begin = 0, end = 0;
  unsigned first = 0;
  if (!rt.find(t, g, begin, end, first)) return;
  const int m0 = begin + (int)(t - first) * 32, n0 = (int)(id % strips) * 16 * NB;
  if (end - m0 <= 16) {
    rows_tile<1, NB, kTB, U>(red, p, ep, g, m0, end, n0, wave, lane);
  } else {
    rows_tile<2, NB, kTB, U>(red, p, ep, g, m0, min(end, m0 + 32), n0, wave, lane);
  }
}

template <int NB, int U>
hipError_t launch(const GroupedProblem& p, const Epilogue& e, hipStream_t s) {
  const int64_t strips = ((int64_t)p.N + 16 * NB - 1) / (16 * NB);
  const int64_t cap = most_row_tiles(p.rows, p.groups, 32);
  if (cap * strips > 0x7fffffff) return hipErrorInvalidConfiguration;
  const dim3 grid = tile_grid(cap * strips), block(kWaves * 64);
  if (p.tb) {
    hipLaunchKernelGGL((grouped_rows_kernel<NB, true, U>), grid, block, 0, s, p, e, (int)strips,
                       (unsigned)cap);
  } else {
    hipLaunchKernelGGL((grouped_rows_kernel<NB, false, U>), grid, block, 0, s, p, e, (int)strips,
                       (unsigned)cap);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_rows(const GroupedProblem& p, const Epilogue& e, hipStream_t s) {
  if (p.N <= 16) return launch<1, 4>(p, e, s);
  if (p.N <= 32 || p.tb) return launch<2, 4>(p, e, s);
  return launch<4, 2>(p, e, s);
}

}  // namespace gemmf32
