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

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace

hipError_t launch_grouped(const GroupedProblem& call, const Epilogue& e, hipStream_t s) {
  GroupedProblem p = call;
  if (p.rows_a == 0) p.K = 0;   // every row of A is outside: empty sums
  // 16-byte copies need whole chunks of both operands inside: bases, pitches
  // and strides of 16 bytes, and the contiguous sizes multiples of 4
  const bool wide = aligned16(p.A) && aligned16(p.B) && p.lda % 4 == 0 && p.ldb % 4 == 0 &&
                    (p.groups == 1 || p.sb % 4 == 0) && p.K % 4 == 0 && (p.tb || p.N % 4 == 0);
  // few rows in a group, few columns, or few sums: bound by one read of B or of A,
  // or by the latency of a tile (16 groups of 32, 1024 x 1024: 27 us against 43 us
  // for the tiles; of 64: 34 against 43; of 96: 49 against 43; 64 groups of 48: 130
  // against 77)
  const int64_t busy = p.rows < p.groups ? p.rows : p.groups, sums = (int64_t)p.rows * p.N;
  if (p.N <= 64 || p.rows <= 32 * busy || (p.rows <= 64 * busy && sums <= 1 << 20) || sums <= 1 << 18)
    return launch_grouped_rows(p, e, s);
  // about how many 128 x 128 and 64 x 64 tiles
  const int64_t tiles =
      ((int64_t)p.rows / 128 + p.groups / 2) * (((int64_t)p.N + 127) / 128);
  const int64_t tiles64 = ((int64_t)p.rows / 64 + p.groups / 2) * (((int64_t)p.N + 63) / 64);
  if (wide) {
    // tiles that leave three CUs in eight idle (2 groups of 512, 4096 x 512: 60 us
    // against 86 us for the tiles; 3 of 512, 1024 x 512, half as many tiles more: 30
    // against 26)
    if (tiles64 <= kCus / 8 * 5) return launch_grouped_rows(p, e, s);
    // 64 x 64 tiles, four workgroups a CU, below a round of the CUs (21 groups of 261,
    // 1280 x 384: 71 us against 87 us in mixed tiles), where the second round would be
    // neither nearly empty nor full (8 of 512, 1024 x 1280: 111 against 123), and for
    // groups that fill few of the rows of 128 (64 of 128, 512 x 768: 78 against 86)
    const bool small = tiles < kCus || (tiles >= kCus / 4 * 5 && tiles < 2 * kCus) ||
                       p.rows <= 192 * (int64_t)p.groups;
    if (!small) return launch_mixed(p, e, s);
    return p.tb ? launch_even<64, 64, 32, 32, 32, true, 4, 4>(p, e, s)
                : launch_even<64, 64, 32, 32, 32, false, 4, 4>(p, e, s);
  }
  // copies of single floats.  B stored N x K: below four rounds of 128 x 128 tiles the
  // kernel for few rows, whose 16-byte loads fit any row (3 groups of 500, 1501 x 1001:
  // 56 us against 75 us in 64 x 64 tiles; 16 of 437, 515 x 1027: 92 against 136 in tiles
  // of 128; 4 of 3000, 1027 x 1025: 287 against 338; 2 of 4096, 2047 x 1001: 392
  // against 335; 8 of 2048, 2049 x 2047: 1978 against 1314).
  if (p.tb)
    return tiles < 4 * (int64_t)kCus ? launch_grouped_rows(p, e, s)
                                     : launch_even<128, 128, 16, 64, 32, true, 1, 2>(p, e, s);
  // Stored K x N below four rounds of 64 x 64 tiles, where the last round counts for
  // most (13 of 161, 769 x 1001: 61 against 68 us; 16 of 200, 511 x 1025: 58 against
  // 72; 2 of 1300, 1501 x 1001: 112 against 122; 8 of 250, 513 x 1023, two whole rounds:
  // 44 against 37; 8 of 512, 2049 x 1023, four: 235 against 214); then those, and 128 x
  // 128 tiles where they make two rounds (8 x 1000 x 1023 x 2047: 333 us against 452)
  if (tiles64 < 4 * (int64_t)kCus) return launch_grouped_rows(p, e, s);
  return tiles >= 2 * (int64_t)kCus ? launch_even<128, 128, 16, 64, 32, false, 1, 2>(p, e, s)
                                    : launch_even<64, 64, 16, 32, 32, false, 1, 4>(p, e, s);
}

}  // namespace gemmf32
