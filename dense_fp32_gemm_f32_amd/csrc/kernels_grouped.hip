// Products whose rows belong to different weights (gfx950): for every place i
// of group g, C[ic(i)] = act(alpha s_g A[ia(i)] op(B_g) + beta C[ic(i)] + bias_g).
//
// The group sizes are known on the device only, so the grid covers the most row
// tiles that the places can need; each workgroup finds its tile from the
// offsets (a scan of 64 groups in a wave) and ends at once if there is none.
#include "grouped_routes.h"
#include "grouped_tile.h"

namespace gemmf32 {
namespace {

using namespace grouped;

// kWaves waves copy, the first (BM / WM) (BN / WN) of them multiply.
template <int BM, int BN, int BK, int WM, int WN, bool kTB, int V,
          int kWaves = (BM / WM) * (BN / WN)>
__device__ __forceinline__ void grouped_tile(float* pool, const int* row_a, const int* row_c,
                                             bool absent, const GroupedProblem& p,
                                             const Epilogue& ep, int g, int n0, int wave,
                                             int lane) {
  const float* B = p.B + g * p.sb;
  Source<BK, Operand<BM, BK, kWaves, true, V>, Operand<BN, BK, kWaves, kTB, V>> src(
      p.lda, p.ldb, p.K, wave, lane);
  src.a.init_kc(p.A, p.lda, wave, lane, [&](int r) { return max(row_a[r], 0); });
  if constexpr (kTB) {
    src.b.init_kc(B, p.ldb, wave, lane, [&](int r) { return r < p.N - n0 ? n0 + r : 0; });
  } else {
    src.b.init_rc(B, p.ldb, n0, p.N, wave, lane);
  }
  floatx16 acc[WM / 32][WN / 32];
  k_loop<BM, BN, BK, WM, WN>(pool, src, wave, lane, acc);
  if (kWaves > (BM / WM) * (BN / WN) && wave >= (BM / WM) * (BN / WN)) return;
  const int row0 = (wave % (BM / WM)) * WM;
  if (absent) {   // rows whose index is outside count as zeros
#pragma unroll
    for (int i = 0; i < WM / 32; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (row_a[row0 + 32 * i + 4 * (lane >> 5) + 8 * (r >> 2) + (r & 3)] < 0)
#pragma unroll
          for (int j = 0; j < WN / 32; ++j) acc[i][j][r] = 0.f;
  }
  const float scale = p.gscale ? p.gscale[g] : 1.f;
  Epilogue e = ep;
  if (e.bias) e.bias += g * p.sbias;
  store_rows(acc, p.C, p.ldc, p.N, e, scale, row_c, row0, n0 + (wave / (BM / WM)) * WN, lane);
}

// A workgroup's tile and its rows: what both kernels do before their tiles.
struct Place {
  int g, m0, n0, end;   // group, first place and column, end of the group
  bool absent;          // some row of A is outside its matrix
};

// The rows of A and C of the places m0 .. m0 + BM - 1, into LDS.
template <int BM>
__device__ __forceinline__ void find_rows(const GroupedProblem& p, Place& at, int* row_a,
                                          int* row_c) {
  const Gather ga{p.ia, p.rows_a}, gc{p.ic, p.rows_c};
  int outside = 0;
  if ((int)threadIdx.x < BM) {
    const int a = ga.at(at.m0 + threadIdx.x, at.end), c = gc.at(at.m0 + threadIdx.x, at.end);
    row_a[threadIdx.x] = a;
    row_c[threadIdx.x] = c;
    outside = a < 0 && c >= 0;
  }
  at.absent = __syncthreads_or(outside);
}

// 16-byte copies, in mixed tiles of 8 waves; four of them multiply a quarter.
// (64 x 128 tiles for a group's last 64 places or fewer made no shape faster and
// 8192 x 1024 x 1408 slower, 228 against 197 us.)
template <bool kTB>
__global__ void __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(4)))
    grouped_mixed_kernel(GroupedProblem p, Epilogue ep, int tiles_n, unsigned cap) {
  constexpr int BM = 128, BN = 128, BK = 32;
  __shared__ __attribute__((aligned(16))) float pool[2 * (BM + BN) * BK];
  __shared__ int row_a[BM], row_c[BM];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowTiles rt{p.offsets, p.groups, p.rows, BM, lane, cap, 0};
  const MixedTile mt = mixed_tile(rt.total(), tiles_n);
  if (!mt.any) return;
  Place at{};
  int begin = 0;
  unsigned first = 0;
  if (!rt.find((unsigned)mt.tm, at.g, begin, at.end, first)) return;
  at.m0 = begin + (mt.tm - (int)first) * BM + mt.m_off;
  at.n0 = mt.tn * BN + mt.n_off;
  if (at.m0 >= at.end || at.n0 >= p.N) return;
  find_rows<BM>(p, at, row_a, row_c);
  if (mt.quarter) {
    grouped_tile<64, 64, BK, 32, 32, kTB, 4, 8>(pool, row_a, row_c, at.absent, p, ep, at.g, at.n0,
                                                wave, lane);
  } else {
    grouped_tile<128, 128, BK, 64, 32, kTB, 4>(pool, row_a, row_c, at.absent, p, ep, at.g, at.n0,
                                               wave, lane);
  }
}

// Tiles of one size, BM x BN in waves of WM x WN; copies of V floats (1: for any
// pitch and alignment).
template <int BM, int BN, int BK, int WM, int WN, bool kTB, int V, int kMinWaves>
__global__ void __launch_bounds__((BM / WM) * (BN / WN) * 64)
    __attribute__((amdgpu_waves_per_eu(kMinWaves)))
    grouped_even_kernel(GroupedProblem p, Epilogue ep, int tiles_n, unsigned cap) {
  __shared__ __attribute__((aligned(16))) float pool[2 * (BM + BN) * BK];
  __shared__ int row_a[BM], row_c[BM];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  RowTiles rt{p.offsets, p.groups, p.rows, BM, lane, cap, 0};
  const unsigned total = rt.total();
  const int pos = xcd_position(tile_id(), total * (unsigned)tiles_n);
  if (pos < 0) return;
  int tm, tn, begin = 0;
  tile_coords(pos, (int)total, tiles_n, tm, tn);
  Place at{};
  unsigned first = 0;
  if (!rt.find((unsigned)tm, at.g, begin, at.end, first)) return;
  at.m0 = begin + (tm - (int)first) * BM;
  at.n0 = tn * BN;
  find_rows<BM>(p, at, row_a, row_c);
  grouped_tile<BM, BN, BK, WM, WN, kTB, V>(pool, row_a, row_c, at.absent, p, ep, at.g, at.n0, wave,
                                           lane);
}

hipError_t launch_mixed(const GroupedProblem& p, const Epilogue& e, hipStream_t s) {
  const int64_t tiles_n = ((int64_t)p.N + 127) / 128;
  const int64_t cap = most_row_tiles(p.rows, p.groups, 128);
  if (cap * tiles_n + 3 * kCus > 0x7fffffff) return hipErrorInvalidConfiguration;
  const dim3 grid = tile_grid(cap * tiles_n + 3 * kCus);
  if (p.tb) {
    hipLaunchKernelGGL((grouped_mixed_kernel<true>), grid, dim3(512), 0, s, p, e, (int)tiles_n,
                       (unsigned)cap);
  } else {
    hipLaunchKernelGGL((grouped_mixed_kernel<false>), grid, dim3(512), 0, s, p, e, (int)tiles_n,
                       (unsigned)cap);
  }
  return hipGetLastError();
}

template <int BM, int BN, int BK, int WM, int WN, bool kTB, int V, int kMinWaves>
hipError_t launch_even(const GroupedProblem& p, const Epilogue& e, hipStream_t s) {
  const int64_t tiles_n = ((int64_t)p.N + BN - 1) / BN;
  const int64_t cap = most_row_tiles(p.rows, p.groups, BM);
  if (cap * tiles_n > 0x7fffffff) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((grouped_even_kernel<BM, BN, BK, WM, WN, kTB, V, kMinWaves>),
                     tile_grid(cap * tiles_n), dim3((BM / WM) * (BN / WN) * 64), 0, s, p, e,
                     (int)tiles_n, (unsigned)cap);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped(const GroupedProblem& call, const Epilogue& e, hipStream_t s) {
  GroupedProblem p = call;
  if (p.rows_a == 0) p.K = 0;   // every row of A is outside: empty sums
  switch (product_kernel(p)) {
    case ProductKernel::Rows:
      return launch_grouped_rows(p, e, s);
    case ProductKernel::Mixed:
      return launch_mixed(p, e, s);
    case ProductKernel::Even64:
      return p.tb ? launch_even<64, 64, 32, 32, 32, true, 4, 4>(p, e, s)
                  : launch_even<64, 64, 32, 32, 32, false, 4, 4>(p, e, s);
    case ProductKernel::Even64Single:   // stored K x N only
      return launch_even<64, 64, 16, 32, 32, false, 1, 4>(p, e, s);
    case ProductKernel::Even128Single:
      return p.tb ? launch_even<128, 128, 16, 64, 32, true, 1, 2>(p, e, s)
                  : launch_even<128, 128, 16, 64, 32, false, 1, 2>(p, e, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace gemmf32
