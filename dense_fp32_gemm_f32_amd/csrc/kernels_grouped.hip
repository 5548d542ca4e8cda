// Products whose rows belong to different weights (gfx950): for every place i
// of group g, C[ic(i)] = act(alpha s_g A[ia(i)] op(B_g) + beta C[ic(i)] + bias_g).
//
// The group sizes are known on the device only, so the grid covers the most row
// tiles that the places can need; each workgroup finds its tile from the
// offsets (a scan of 64 groups in a wave) and ends at once if there is none.
#include "grouped_tile.h"

namespace gemmf32 {
namespace {

using namespace grouped;

// The update of a wave's blocks, rows of C through row_c (LDS; -1: not
// written).  The plain product stores the sums themselves.
template <int KFM, int KFN>
__device__ __forceinline__ void store_rows(const floatx16 (&acc)[KFM][KFN],
                                           const GroupedProblem& p, const Epilogue& ep,
                                           float scale, const int* row_c, int row0, int col0,
                                           int lane) {
  const int lr = lane & 31, lk = lane >> 5;
  const bool direct = scale == 1.f && ep.alpha == 1.f && ep.beta == 0.f && !ep.bias && ep.act == 0;
#pragma unroll
  for (int i = 0; i < KFM; ++i) {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int c = row_c[row0 + 32 * i + 4 * lk + 8 * (r >> 2) + (r & 3)];
      if (c < 0) continue;
      float* out = p.C + c * p.ldc;
#pragma unroll
      for (int j = 0; j < KFN; ++j) {
        const int col = col0 + 32 * j + lr;
        if (col < p.N)
          out[col] = direct ? acc[i][j][r]
                            : epilogue_apply(ep, scale * acc[i][j][r], out + col, col);
      }
    }
  }
}

template <int BM, int BN, int BK, int WM, int WN, bool kTB, int V>
__device__ __forceinline__ void grouped_tile(float* pool, const int* row_a, const int* row_c,
                                             const GroupedProblem& p, const Epilogue& ep, int g,
                                             int n0, int wave, int lane) {
  constexpr int kWaves = (BM / WM) * (BN / WN);
  const float* B = p.B + g * p.sb;
  Operand<BM, BK, kWaves, true, V> opa;
  Operand<BN, BK, kWaves, kTB, V> opb;
  opa.init_kc(p.A, p.lda, wave, lane, [&](int r) { return row_a[r]; });
  if constexpr (kTB) {
    opb.init_kc(B, p.ldb, wave, lane, [&](int r) { return r < p.N - n0 ? n0 + r : -1; });
  } else {
    opb.init_rc(B, p.ldb, n0, p.N, wave, lane);
  }
  floatx16 acc[WM / 32][WN / 32];
  k_loop<BM, BN, BK, WM, WN>(pool, opa, opb, Gather{}, Gather{}, 0, p.lda, p.ldb, p.K, wave, lane,
                             acc);
  const float scale = p.gscale ? p.gscale[g] : 1.f;
  Epilogue e = ep;
  if (e.bias) e.bias += g * p.sbias;
  store_rows(acc, p, e, scale, row_c, (wave % (BM / WM)) * WM, n0 + (wave / (BM / WM)) * WN, lane);
}

template <int BM, int BN, int BK, int WM, int WN, bool kTB, int V, int kMinWaves>
__global__ void __launch_bounds__((BM / WM) * (BN / WN) * 64)
    __attribute__((amdgpu_waves_per_eu(kMinWaves)))
    grouped_kernel(GroupedProblem p, Epilogue ep, int tiles_n, unsigned cap) {
  __shared__ __attribute__((aligned(16))) float pool[2 * (BM + BN) * BK];
  __shared__ int row_a[BM], row_c[BM];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  RowTiles rt{p.offsets, p.groups, p.rows, BM, lane, cap, 0};
  const unsigned total = rt.total(), tiles = total * (unsigned)tiles_n;
  // each XCD takes a contiguous range of the tiles that there are
  const unsigned id = tile_id();
  const unsigned x = id % kNumXcd, q = tiles / kNumXcd, rem = tiles % kNumXcd;
  if (id / kNumXcd >= q + (x < rem ? 1u : 0u)) return;
  int tm, tn;
  tile_coords((int)(x * q + min(x, rem) + id / kNumXcd), (int)total, tiles_n, tm, tn);
  int g = 0, begin = 0, end = 0;
  unsigned first = 0;
  if (!rt.find((unsigned)tm, g, begin, end, first)) return;
  const int m0 = begin + (tm - (int)first) * BM;
  const Gather ga{p.ia, p.rows_a}, gc{p.ic, p.rows_c};
  if (tid < BM) {
    row_a[tid] = ga.at(m0 + tid, end);
    row_c[tid] = gc.at(m0 + tid, end);
  }
  __syncthreads();
  grouped_tile<BM, BN, BK, WM, WN, kTB, V>(pool, row_a, row_c, p, ep, g, tn * BN, wave, lane);
}

template <int BM, int BN, int BK, int WM, int WN, int V, int kMinWaves>
hipError_t launch(const GroupedProblem& p, const Epilogue& e, hipStream_t s) {
  const int64_t tiles_n = ((int64_t)p.N + BN - 1) / BN;
  const int64_t cap = most_row_tiles(p.rows, p.groups, BM);
  if (cap * tiles_n > 0x7fffffff) return hipErrorInvalidConfiguration;
  const dim3 grid = tile_grid(cap * tiles_n), block((BM / WM) * (BN / WN) * 64);
  if (p.tb) {
    hipLaunchKernelGGL((grouped_kernel<BM, BN, BK, WM, WN, true, V, kMinWaves>), grid, block, 0, s,
                       p, e, (int)tiles_n, (unsigned)cap);
  } else {
    hipLaunchKernelGGL((grouped_kernel<BM, BN, BK, WM, WN, false, V, kMinWaves>), grid, block, 0, s,
                       p, e, (int)tiles_n, (unsigned)cap);
  }
  return hipGetLastError();
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace

hipError_t launch_grouped(const GroupedProblem& p, const Epilogue& e, hipStream_t s) {
  // few rows in a group, or few columns: bound by one read of B or of A
  if (p.rows <= 24 * (int64_t)p.groups || p.rows <= 64 || p.N <= 64)
    return launch_grouped_rows(p, e, s);
  // 16-byte copies need whole chunks of both operands inside: bases, pitches
  // and strides of 16 bytes, and the contiguous sizes multiples of 4
  const bool wide = aligned16(p.A) && aligned16(p.B) && p.lda % 4 == 0 && p.ldb % 4 == 0 &&
                    (p.groups == 1 || p.sb % 4 == 0) && p.K % 4 == 0 && (p.tb || p.N % 4 == 0);
  if (!wide) return launch<64, 64, 16, 32, 32, 1, 4>(p, e, s);
  if ((int64_t)p.rows * p.N < (INT64_C(1) << 20)) return launch<64, 64, 32, 32, 32, 4, 4>(p, e, s);
  return launch<128, 128, 32, 64, 32, 4, 2>(p, e, s);
}

}  // namespace gemmf32
