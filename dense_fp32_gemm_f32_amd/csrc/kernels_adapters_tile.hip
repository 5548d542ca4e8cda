// The shared projection with low-rank adapters added to its tiles (gfx950): Y = X
// op(W) + bias + H[place] op(U_g) for the rows that have an adapter.
//
// H is there already (H[place] = s_g X[row] op(D_g)), with a map from rows to their
// places and adapters.  A workgroup computes its tile of X op(W) and then, for
// each adapter among its rows, the K loop goes on over the adapter's rank, its
// copies already on the way: A's rows are H's where the row has that adapter and
// zeros elsewhere.  Rows in a batch come request by request, so a tile meets one
// or two adapters, and each costs it one K-tile or two, where a product of its own
// would read and write Y again.
//
// The map is written by the rows that have an adapter only and never cleared: an
// entry counts if its place names this row and lies in its adapter's places.
#include "grouped_tile.h"

namespace gemmf32 {
namespace {

using namespace grouped;

constexpr int kMaxRank = 64;
constexpr int kBK = 32;
// rows of H for rows of another adapter, or none
static __device__ __attribute__((aligned(16))) const float kZeroRank[kMaxRank] = {};

// The smallest adapter above `after` in adapter[0 .. BM - 1], kMaxGroups if there
// is none; every wave finds it alone.
template <int BM>
__device__ __forceinline__ int next_adapter(const int* adapter, int after, int lane) {
  int v = kMaxGroups;
#pragma unroll
  for (int i = 0; i < BM; i += 64) {
    const int a = adapter[i + lane];
    if (a > after) v = min(v, a);
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v = min(v, __shfl_xor(v, d));
  return __builtin_amdgcn_readfirstlane(v);
}

// The K loop's copies: X and W, then H and U_g for each adapter g of the tile.
template <int BM, int BN, int kWaves, bool kTB>
struct AdapterSource {
  using OpA = Operand<BM, kBK, kWaves, true, 4>;
  using OpB = Operand<BN, kBK, kWaves, kTB, 4>;
  OpA a;
  OpB b;
  const AdapterProblem& p;
  const int *place, *adapter;   // LDS, of the tile's rows
  int n0, wave, lane;
  int base, per, all;           // K-tiles of the projection, of an adapter, of the tile
  int g = -1, end = 0;          // the adapter copied from, and its first K-tile past the end
  int64_t lda, ldb;
  int k0 = 0, k_end;

  __device__ __forceinline__ AdapterSource(const AdapterProblem& p_, const int* place_,
                                           const int* adapter_, int m0, int n0_, int wave_,
                                           int lane_)
      : p(p_), place(place_), adapter(adapter_), n0(n0_), wave(wave_), lane(lane_) {
    base = end = (p.K + kBK - 1) / kBK;
    per = (p.R + kBK - 1) / kBK;
    all = base;
    for (int x = next_adapter<BM>(adapter, -1, lane); x < kMaxGroups;
         x = next_adapter<BM>(adapter, x, lane))
      all += per;
    a.init_kc(p.X, p.ldx, wave, lane, [&](int r) { return min(m0 + r, p.M - 1); });
    init_b(p.W, p.ldw);
    lda = p.ldx;
    ldb = p.ldw;
    k_end = p.K;
  }
  __device__ __forceinline__ void init_b(const float* B, int64_t ld) {
    if constexpr (kTB) {
      b.init_kc(B, ld, wave, lane, [&](int r) { return r < p.N - n0 ? n0 + r : 0; });
    } else {
      b.init_rc(B, ld, n0, p.N, wave, lane);
    }
  }
  __device__ __forceinline__ int tiles() const { return all; }
  __device__ __forceinline__ void seek(int t) {
    if (t >= all) return;   // the last K-tile again
    if (t == end) {         // on to the next adapter
      const int x = g = next_adapter<BM>(adapter, g, lane);
      end += per;
      a.init_rows(wave, lane, [&](int r, int k) {
        return adapter[r] == x ? p.H + place[r] * p.ldh + k : kZeroRank + k;
      });
      init_b(p.U + x * p.su, p.ldu);
      lda = p.ldh;
      ldb = p.ldu;
      k_end = p.R;
    }
    k0 = (g < 0 ? t : t - (end - per)) * kBK;
  }
  __device__ __forceinline__ void copy(float* la, float* lb, int idx) const {
    if (idx < OpA::kCopies) {
      a.copy(idx, la, lda, k0, k_end, 0, wave, lane);
    } else {
      b.copy(idx - OpA::kCopies, lb, ldb, k0, k_end, 0, wave, lane);
    }
  }
};

template <int BM, int BN, int WM, int WN, bool kTB>
__device__ __forceinline__ void adapter_tile(float* pool, const int* row, const int* place,
                                             const int* adapter, const AdapterProblem& p, int m0,
                                             int n0, int wave, int lane) {
  AdapterSource<BM, BN, (BM / WM) * (BN / WN), kTB> src(p, place, adapter, m0, n0, wave, lane);
  floatx16 acc[WM / 32][WN / 32];
  k_loop<BM, BN, kBK, WM, WN>(pool, src, wave, lane, acc);
  Epilogue e;
  e.bias = p.bias;
  store_rows(acc, p.Y, p.ldy, p.N, e, 1.f, row, (wave % (BM / WM)) * WM,
             n0 + (wave / (BM / WM)) * WN, lane);
}

// The tile's rows: row of Y (-1 past M), place and adapter (-1 for none).
template <int BM>
__device__ __forceinline__ void find_adapters(const AdapterProblem& p, const int* map, int m0,
                                              int* row, int* place, int* adapter) {
  const int tid = threadIdx.x, m = m0 + tid;
  if (tid < BM) {
    int at = -1, g = -1;
    if (m < p.M) {
      at = map[2 * (int64_t)m];
      g = map[2 * (int64_t)m + 1];
      bool in = at >= 0 && at < p.places && g >= 0 && g < p.groups && p.order[at] == m;
      if (in) {
        int b, e;
        group_span(p.offsets, g, p.places, b, e);
        in = at >= b && at < e;
      }
      if (!in) g = -1;
    }
    row[tid] = m < p.M ? m : -1;
    place[tid] = at;
    adapter[tid] = g;
  }
  __syncthreads();
}

// Mixed tiles; the last row tile of at most 64 rows is 64 x 128.
template <bool kTB>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2)))
    adapters_mixed_kernel(AdapterProblem p, const int* __restrict__ map, int tiles_m, int tiles_n) {
  constexpr int BM = 128, BN = 128;
  __shared__ __attribute__((aligned(16))) float pool[2 * (BM + BN) * kBK];
  __shared__ int row[BM], place[BM], adapter[BM];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const MixedTile mt = mixed_tile((unsigned)tiles_m, tiles_n);
  if (!mt.any) return;
  const int m0 = mt.tm * BM + mt.m_off, n0 = mt.tn * BN + mt.n_off;
  if (m0 >= p.M || n0 >= p.N) return;
  find_adapters<BM>(p, map, m0, row, place, adapter);
  if (mt.quarter) {
    adapter_tile<64, 64, 32, 32, kTB>(pool, row, place, adapter, p, m0, n0, wave, lane);
  } else if (p.M - m0 <= 64) {
    adapter_tile<64, 128, 32, 64, kTB>(pool, row, place, adapter, p, m0, n0, wave, lane);
  } else {
    adapter_tile<128, 128, 64, 64, kTB>(pool, row, place, adapter, p, m0, n0, wave, lane);
  }
}

// 64 x 64 tiles, for less than a round of the larger ones.
template <bool kTB>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(4)))
    adapters_small_kernel(AdapterProblem p, const int* __restrict__ map, int tiles_m, int tiles_n) {
  constexpr int BM = 64, BN = 64;
  __shared__ __attribute__((aligned(16))) float pool[2 * (BM + BN) * kBK];
  __shared__ int row[BM], place[BM], adapter[BM];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pos = xcd_position(tile_id(), (unsigned)(tiles_m * tiles_n));
  if (pos < 0) return;
  int tm, tn;
  tile_coords(pos, tiles_m, tiles_n, tm, tn);
  find_adapters<BM>(p, map, tm * BM, row, place, adapter);
  adapter_tile<64, 64, 32, 32, kTB>(pool, row, place, adapter, p, tm * BM, tn * BN, wave, lane);
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace

bool adapters_tiles(const AdapterProblem& p) {
  // 16-byte copies of every operand; and so few adapters that a tile whose rows
  // have them all takes at most half as long again
  return p.R <= kMaxRank && p.R % 4 == 0 && p.K % 4 == 0 && (p.trans || p.N % 4 == 0) &&
         p.ldx % 4 == 0 && p.ldw % 4 == 0 && p.ldu % 4 == 0 && p.ldh % 4 == 0 &&
         (p.groups == 1 || p.su % 4 == 0) && aligned16(p.X) && aligned16(p.W) && aligned16(p.U) &&
         aligned16(p.H) && (int64_t)p.groups * ((p.R + kBK - 1) / kBK) * 2 <= p.K / kBK;
}

hipError_t launch_adapters_tiles(const AdapterProblem& p, const int* map, hipStream_t s) {
  const int64_t tiles_m = ((int64_t)p.M + 127) / 128, tiles_n = ((int64_t)p.N + 127) / 128;
  if (tiles_m * tiles_n + 3 * kCus > 0x7fffffff) return hipErrorInvalidConfiguration;
  if (tiles_m * tiles_n < kCus) {
    const int tm = (p.M + 63) / 64, tn = (p.N + 63) / 64;
    const dim3 grid = tile_grid((int64_t)tm * tn);
    if (p.trans) {
      hipLaunchKernelGGL((adapters_small_kernel<true>), grid, dim3(256), 0, s, p, map, tm, tn);
    } else {
      hipLaunchKernelGGL((adapters_small_kernel<false>), grid, dim3(256), 0, s, p, map, tm, tn);
    }
    return hipGetLastError();
  }
  const dim3 grid = tile_grid(tiles_m * tiles_n + 3 * kCus);
  if (p.trans) {
    hipLaunchKernelGGL((adapters_mixed_kernel<true>), grid, dim3(256), 0, s, p, map, (int)tiles_m,
                       (int)tiles_n);
  } else {
    hipLaunchKernelGGL((adapters_mixed_kernel<false>), grid, dim3(256), 0, s, p, map, (int)tiles_m,
                       (int)tiles_n);
  }
  return hipGetLastError();
}

}  // namespace gemmf32
