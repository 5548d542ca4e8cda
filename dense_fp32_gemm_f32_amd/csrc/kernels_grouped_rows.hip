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
  if (p.map && n0 == 0 && (int)threadIdx.x < min(BM, end - m0)) {
    const int i = m0 + threadIdx.x, r = p.ia ? p.ia[i] : i;
    if (r >= 0 && r < p.rows_a) {
      p.map[2 * (int64_t)r] = i;
      p.map[2 * (int64_t)r + 1] = g;
    }
  }
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

template <int RM, int NB, bool kTB, int U>
__global__ void __launch_bounds__(kWaves * 64)
    grouped_rows_kernel(GroupedProblem p, Epilogue ep, int strips, unsigned cap) {
  constexpr int BM = 16 * RM;
  __shared__ float red[kWaves * BM * 16 * NB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  RowTiles rt{p.offsets, p.groups, p.rows, BM, lane, cap, 0};
  const unsigned total = rt.total();
  const unsigned id = tile_id(), t = id / strips;
  if (t >= total) return;
  int g = 0, begin = 0, end = 0;
  unsigned first = 0;
  if (!rt.find(t, g, begin, end, first)) return;
  const int m0 = begin + (int)(t - first) * BM, n0 = (int)(id % strips) * 16 * NB;
  if (RM == 1 || end - m0 <= 16) {
    rows_tile<1, NB, kTB, U>(red, p, ep, g, m0, min(end, m0 + 16), n0, wave, lane);
  } else {
    rows_tile<RM, NB, kTB, U>(red, p, ep, g, m0, min(end, m0 + BM), n0, wave, lane);
  }
}

template <int RM, int NB>
hipError_t launch(const GroupedProblem& p, const Epilogue& e, hipStream_t s) {
  const int64_t strips = ((int64_t)p.N + 16 * NB - 1) / (16 * NB);
  const int64_t cap = most_row_tiles(p.rows, p.groups, 16 * RM);
  if (cap * strips > 0x7fffffff) return hipErrorInvalidConfiguration;
  const dim3 grid = tile_grid(cap * strips), block(kWaves * 64);
  if (p.tb) {
    hipLaunchKernelGGL((grouped_rows_kernel<RM, NB, true, 4>), grid, block, 0, s, p, e, (int)strips,
                       (unsigned)cap);
  } else {
    hipLaunchKernelGGL((grouped_rows_kernel<RM, NB, false, NB == 4 ? 2 : 4>), grid, block, 0, s, p,
                       e, (int)strips, (unsigned)cap);
  }
  return hipGetLastError();
}

template <int RM>
hipError_t launch_strips(const GroupedProblem& p, int nb, const Epilogue& e, hipStream_t s) {
  return nb == 1 ? launch<RM, 1>(p, e, s) : nb == 2 ? launch<RM, 2>(p, e, s)
                                                    : launch<RM, 4>(p, e, s);
}

}  // namespace

hipError_t launch_grouped_rows(const GroupedProblem& p, const Epilogue& e, hipStream_t s) {
  // few columns: 16 places a workgroup, all columns in one strip up to 64 (4096
  // places of 2048, 32 columns: 14 us against 20 us for 32 places)
  if (p.N <= 64) return launch_strips<1>(p, p.N <= 16 ? 1 : p.N <= 32 ? 2 : 4, e, s);
  // few rows in a group: 32 places where groups have more than 10 on average (16
  // groups of 19, 1024 x 1024: 19 against 24 us), else 16 (less LDS: 6 places,
  // 32 x 1024 x 2048: 47 against 51 us); strips as wide as leaves two workgroups a
  // CU (64 groups of one place: 64 columns 43 us, 32 columns 51, 16 columns 59; 8 of
  // 2048 x 1024: 21, 18 and 16 us)
  const int64_t busy = p.rows < p.groups ? p.rows : p.groups;
  const bool two = p.rows > 10 * busy;
  const int64_t tiles = busy * ((p.rows / busy + (two ? 31 : 15)) / (two ? 32 : 16));
  int nb = 4;
  while (nb > 1 && tiles * (((int64_t)p.N + 16 * nb - 1) / (16 * nb)) < 512) nb /= 2;
  return two ? launch_strips<2>(p, nb, e, s) : launch_strips<1>(p, nb, e, s);
}

}  // namespace gemmf32
