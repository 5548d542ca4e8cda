// The gradient of the weights of a grouped product (gfx950): for every group g,
// over its places i, C_g = alpha sum_i A[ia(i)]^T B[ib(i)] + beta C_g.
//
// Both operands have their rows contiguous and are gathered along k (the
// places), so a K-tile's matrix rows are fetched one K-tile ahead of its copies.
// Where C has few tiles, long groups are cut into slices of their places.
#include "grouped_routes.h"
#include "grouped_tile.h"

namespace gemmf32 {
namespace {

using namespace grouped;

// A group's size in its lane, -1 past the last group.
__device__ __forceinline__ int group_size(const int* offsets, int groups, int rows, int lane) {
  if (lane >= groups) return -1;
  int b, e;
  group_span(offsets, lane, rows, b, e);
  return e - b;
}

// The n-th largest of at most 64 groups (equal ones by number), found by each
// wave: bit by bit from the top, the groups that can still be it.  A tile takes as
// long as its group has places, so the longest start first and the shortest fill
// the end (8 uneven groups of 8192 places, 1024 x 2048: 334 -> 292 us); finding it
// costs 3 us in each of many short tiles (32 groups of 32, 1024 x 1024: 42 against 39
// us in the groups' own order).
__device__ __forceinline__ int nth_largest(const int* offsets, int groups, int rows, int n,
                                           int lane) {
  const int mine = group_size(offsets, groups, rows, lane);
  unsigned long long left = __ballot(lane < groups);
  for (int b = 31 - __builtin_clz(rows | 1); b >= 0; --b) {
    const unsigned long long ones = __ballot((mine >> b) & 1) & left;
    const int more = __builtin_popcountll(ones);
    left = n < more ? ones : left & ~ones;
    n -= n < more ? 0 : more;
  }
  const int before = __builtin_popcountll(left & ((1ull << lane) - 1));
  return __builtin_ctzll(__ballot((left >> lane & 1) && before == n));
}

template <int BM, int BN, int BK, int WM, int WN, int V, int kMinWaves>
__global__ void __launch_bounds__((BM / WM) * (BN / WN) * 64)
    __attribute__((amdgpu_waves_per_eu(kMinWaves)))
    grouped_wgrad_kernel(GroupedProblem p, Epilogue ep, int tiles_m, int tiles_n, int slices,
                         float* part) {
  constexpr int kWaves = (BM / WM) * (BN / WN);
  __shared__ __attribute__((aligned(16))) float pool[2 * (BM + BN) * BK];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // the groups' tiles in order of the groups' sizes if those are long, each spread over
  // the XCDs in contiguous ranges, a slice's together
  const unsigned id = tile_id(), tiles = (unsigned)tiles_m * tiles_n, each = tiles * slices;
  if (id >= each * p.groups) return;
  const bool sorted = p.groups <= 64 && p.rows > 32 * p.groups;   // one K-tile each is short
  const int g = sorted ? nth_largest(p.offsets, p.groups, p.rows, (int)(id / each), lane)
                       : (int)(id / each);
  const unsigned at = (unsigned)xcd_contiguous_id((int)(id % each), (int)each);
  const int slice = (int)(at / tiles);
  int tm, tn;
  tile_coords((int)(at % tiles), tiles_m, tiles_n, tm, tn);
  int begin, end;
  group_span(p.offsets, g, p.rows, begin, end);
  if (slices > 1) {   // whole K-tiles of the group's places
    const int64_t len = ((int64_t)(end - begin) + slices * BK - 1) / (slices * BK) * BK;
    begin = (int)min((int64_t)end, begin + slice * len);
    end = (int)min((int64_t)end, begin + len);
  }
  begin = __builtin_amdgcn_readfirstlane(begin);
  end = __builtin_amdgcn_readfirstlane(end);
  // an empty span may begin behind the last place: no index entry to look at
  const bool none = begin == end;
  Source<BK, Operand<BM, BK, kWaves, false, V, true>, Operand<BN, BK, kWaves, false, V, true>> src(
      p.lda, p.ldb, end - begin, wave, lane);
  src.a.init_rc(p.A, p.lda, tm * BM, p.M, wave, lane);
  src.b.init_rc(p.B, p.ldb, tn * BN, p.N, wave, lane);
  src.ga = Gather{none ? nullptr : p.ia, p.rows_a};
  src.gb = Gather{none ? nullptr : p.ib, p.rows_b};
  src.first = begin;
  floatx16 acc[WM / 32][WN / 32];
  k_loop<BM, BN, BK, WM, WN, true>(pool, src, wave, lane, acc);
  const int m0 = tm * BM + (wave % (BM / WM)) * WM, n0 = tn * BN + (wave / (BM / WM)) * WN;
  if (slices > 1) {
    float* C = part + ((int64_t)slice * p.groups + g) * p.M * p.N;
    store_blocks<WM / 32, WN / 32>(acc, C, p.N, p.M, p.N, m0, n0, lane, false, Epilogue{});
  } else {
    store_blocks<WM / 32, WN / 32>(acc, p.C + g * p.sc, p.ldc, p.M, p.N, m0, n0, lane, false, ep);
  }
}

template <int BM, int BN, int BK, int WM, int WN, int V, int kMinWaves>
hipError_t launch(const GroupedProblem& p, const Epilogue& e, int slices, float* part,
                  hipStream_t s) {
  const int64_t tiles_m = ((int64_t)p.M + BM - 1) / BM, tiles_n = ((int64_t)p.N + BN - 1) / BN;
  const int64_t n = tiles_m * tiles_n * slices * p.groups;
  if (n > 0x7fffffff) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((grouped_wgrad_kernel<BM, BN, BK, WM, WN, V, kMinWaves>), tile_grid(n),
                     dim3((BM / WM) * (BN / WN) * 64), 0, s, p, e, (int)tiles_m, (int)tiles_n,
                     slices, part);
  const hipError_t err = hipGetLastError();
  return err != hipSuccess || slices == 1 ? err : launch_wgrad_join(p, e, slices, part, s);
}

}  // namespace

size_t grouped_wgrad_floats(const GroupedProblem& p) {
  if (wgrad_thin(p)) return wgrad_thin_floats(p);
  const int slices = gradient_tiles(p).slices;
  return slices > 1 ? (size_t)slices * p.groups * p.M * p.N : 0;
}

hipError_t launch_grouped_wgrad(const GroupedProblem& p, const Epilogue& e, float* part,
                                hipStream_t s) {
  if (wgrad_thin(p)) return launch_wgrad_thin(p, e, part, s);
  const GradientTiles t = gradient_tiles(p);
  if (t.large)
    return t.wide ? launch<128, 128, 32, 64, 32, 4, 2>(p, e, 1, part, s)
                  : launch<128, 128, 16, 64, 32, 1, 2>(p, e, 1, part, s);
  return t.wide ? launch<64, 64, 32, 32, 32, 4, 4>(p, e, t.slices, part, s)
                : launch<64, 64, 16, 32, 32, 1, 4>(p, e, t.slices, part, s);
}

}  // namespace gemmf32
