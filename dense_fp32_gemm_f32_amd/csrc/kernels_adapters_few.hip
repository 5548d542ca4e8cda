// Low-rank adapters beside a shared projection for few rows (gfx950): Y = X op(W)
// + bias + s_g (X op(D_g)) op(U_g), at most 64 rows.
//
// The projection alone is bound by reading W once, and three dependent launches
// (projection, X op(D), + H op(U)) cost more than that read.  So two launches:
//
//   1. the tiles of X op(W) and of X[order] op(D_g) together, each split over K
//      slices so that they fill the CUs, partial sums to a workspace;
//   2. for every row and 256 columns: the row's place and adapter, H[place] = s_g
//      times the sum of its partial sums, then Y = the sum of the projection's
//      partial sums + bias + H[place] op(U_g), a dot product of R terms for each
//      element; the first column blocks write H.
//
// The slices are added in order, so repeats give the same bits.  (32 rows, 2048 x
// 2048, rank 16, 8 adapters: 10.5 + 6 us, against 52 us for the projection by
// gemm_f32_fused, whose 32 tiles leave most CUs idle, and two grouped products.)
#include "grouped_rows.h"

namespace gemmf32 {
namespace {

using namespace grouped;

constexpr int kWaves = 8;
constexpr int kMaxRows = 64, kMaxRank = 128;
constexpr int kMaxSlices = 16;

struct FewPlan {
  int strips, row_tiles;      // the projection's tiles
  int strips_r, places_tiles; // the adapters' tiles (an upper bound)
  int slices, kslice;
};

template <int RM, int NB, bool kTB, class RowAt>
__device__ __forceinline__ void partial_tile(float* red, const AdapterProblem& p, RowAt row_at,
                                             const float* B, int64_t ldb, int N, int n0, int k0,
                                             int k_len, float* out, int rows) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  rows_product<kWaves, RM, NB, kTB, 2, false>(red, p.X + k0, p.ldx, row_at,
                                              B + (kTB ? (int64_t)k0 : (int64_t)k0 * ldb), ldb, N,
                                              n0, k_len, wave, lane);
  constexpr int BN = 16 * NB;
  for (int x = threadIdx.x; x < 16 * RM * BN; x += kWaves * 64) {
    const int r = x / BN, col = n0 + x % BN;
    if (r < rows && col < N) out[(int64_t)r * N + col] = rows_sum<kWaves, RM, NB>(red, x);
  }
}

template <bool kTB, int NB>
__global__ void __launch_bounds__(kWaves * 64)
    adapters_few_kernel(AdapterProblem p, FewPlan pl, float* part, float* hpart) {
  __shared__ float red[kWaves * 32 * 16 * NB];
  const int base = pl.strips * pl.row_tiles * pl.slices;
  int id = (int)blockIdx.x;
  if (id < base) {
    const int slice = id / (pl.strips * pl.row_tiles);
    id -= slice * pl.strips * pl.row_tiles;
    const int m0 = (id / pl.strips) * 32, n0 = (id % pl.strips) * 16 * NB;
    const int rows = min(32, p.M - m0), k0 = slice * pl.kslice, k_len = min(pl.kslice, p.K - k0);
    float* out = part + ((int64_t)slice * p.M + m0) * p.N;
    auto row_at = [&](int i) { return i < rows ? m0 + i : -1; };
    if (rows <= 16) {
      partial_tile<1, NB, kTB>(red, p, row_at, p.W, p.ldw, p.N, n0, k0, k_len, out, rows);
    } else {
      partial_tile<2, NB, kTB>(red, p, row_at, p.W, p.ldw, p.N, n0, k0, k_len, out, rows);
    }
    return;
  }
  id -= base;
  const int per_slice = pl.strips_r * pl.places_tiles;
  const int slice = id / per_slice;
  id -= slice * per_slice;
  RowTiles rt{p.offsets, p.groups, p.places, 32, (int)(threadIdx.x & 63),
              (unsigned)pl.places_tiles, 0};
  const unsigned t = (unsigned)(id / pl.strips_r);
  if (t >= rt.total()) return;
  int g = 0, begin = 0, end = 0;
  unsigned first = 0;
  if (!rt.find(t, g, begin, end, first)) return;
  const int i0 = begin + (int)(t - first) * 32, n0 = (id % pl.strips_r) * 16;
  const int rows = min(32, end - i0), k0 = slice * pl.kslice, k_len = min(pl.kslice, p.K - k0);
  float* out = hpart + ((int64_t)slice * p.places + i0) * p.R;
  auto row_at = [&](int i) {
    if (i >= rows) return -1;
    const int r = p.order[i0 + i];
    return r >= 0 && r < p.M ? r : -1;
  };
  const float* D = p.D + g * p.sd;
  if (rows <= 16) {
    partial_tile<1, 1, kTB>(red, p, row_at, D, p.ldd, p.R, n0, k0, k_len, out, rows);
  } else {
    partial_tile<2, 1, kTB>(red, p, row_at, D, p.ldd, p.R, n0, k0, k_len, out, rows);
  }
}

// One row of Y and 256 of its columns.
template <bool kTB>
__global__ void __launch_bounds__(256)
    adapters_join_kernel(AdapterProblem p, int slices, const float* __restrict__ part,
                         const float* __restrict__ hpart) {
  __shared__ int group_of[kMaxRows];   // of each place
  __shared__ int place;                // the first place that names this row
  __shared__ float h[kMaxRank];
  const int tid = threadIdx.x, m = blockIdx.y;
  const int n = blockIdx.x * 256 + tid;
  // the projection's partial sums do not wait for the place
  float sum = 0.f;
  if (n < p.N) {
    float v[kMaxSlices];
#pragma unroll
    for (int s = 0; s < kMaxSlices; ++s)
      v[s] = s < slices ? part[((int64_t)s * p.M + m) * p.N + n] : 0.f;
    sum = v[0];
#pragma unroll
    for (int s = 1; s < kMaxSlices; ++s) sum += v[s];
    if (p.bias) sum += p.bias[n];
  }
  if (tid < kMaxRows) group_of[tid] = kMaxGroups;
  if (tid == 0) place = kMaxRows;
  __syncthreads();
  for (int g = tid; g < p.groups; g += 256) {
    int b, e;
    group_span(p.offsets, g, p.places, b, e);
    for (int i = b; i < e; ++i) atomicMin(&group_of[i], g);
  }
  __syncthreads();
  if (tid < p.places && group_of[tid] < kMaxGroups && p.order[tid] == m) atomicMin(&place, tid);
  __syncthreads();
  const int at = place;
  auto h_of = [&](int i, int j) {
    float v = 0.f;
    for (int s = 0; s < slices; ++s) v += hpart[((int64_t)s * p.places + i) * p.R + j];
    return (p.scale ? p.scale[group_of[i]] : 1.f) * v;
  };
  if (blockIdx.x == 0)   // H of the places m, m + M, ..., whatever their rows
    for (int i = m; i < p.places; i += p.M)
      if (group_of[i] < kMaxGroups)
        for (int j = tid; j < p.R; j += 256) p.H[i * p.ldh + j] = h_of(i, j);
  if (at < kMaxRows) {
    const int g = group_of[at];
    for (int j = tid; j < p.R; j += 256) h[j] = h_of(at, j);
    __syncthreads();
    if (n < p.N) {
      const float* u = p.U + g * p.su + (kTB ? n * p.ldu : n);
      const int64_t step = kTB ? 1 : p.ldu;
      float add = 0.f;
      int j = 0;
      for (; j + 8 <= p.R; j += 8) {
        float v[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] = u[(j + x) * step];
#pragma unroll
        for (int x = 0; x < 8; ++x) add += h[j + x] * v[x];
      }
      for (; j < p.R; ++j) add += h[j] * u[j * step];
      sum += add;
    }
  }
  if (n < p.N) p.Y[m * p.ldy + n] = sum;
}

FewPlan plan_few(const AdapterProblem& p) {
  FewPlan pl;
  const int cols = p.trans ? 32 : 64;
  pl.strips = (p.N + cols - 1) / cols;
  pl.row_tiles = (p.M + 31) / 32;
  pl.strips_r = (p.R + 15) / 16;
  pl.places_tiles = (int)most_row_tiles(p.places, p.groups, 32);
  // two workgroups a CU, at least 256 k (two steps of 16 a wave) each
  const int tiles = pl.strips * pl.row_tiles;
  int s = (512 + tiles - 1) / tiles;
  if (s > p.K / 256) s = p.K / 256;
  if (s > kMaxSlices) s = kMaxSlices;
  if (s < 1) s = 1;
  pl.kslice = ((p.K + s - 1) / s + 31) / 32 * 32;
  pl.slices = pl.kslice > 0 ? (p.K + pl.kslice - 1) / pl.kslice : 1;
  return pl;
}

template <bool kTB, int NB>
hipError_t launch(const AdapterProblem& p, const FewPlan& pl, float* part, hipStream_t s) {
  const int64_t blocks =
      (int64_t)pl.slices * ((int64_t)pl.strips * pl.row_tiles + pl.strips_r * pl.places_tiles);
  if (blocks > kGridX || p.N / 256 >= kGridX) return hipErrorInvalidConfiguration;
  float* hpart = part + (size_t)pl.slices * p.M * p.N;
  hipLaunchKernelGGL((adapters_few_kernel<kTB, NB>), dim3((unsigned)blocks), dim3(kWaves * 64), 0,
                     s, p, pl, part, hpart);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL((adapters_join_kernel<kTB>), dim3((unsigned)((p.N + 255) / 256), p.M),
                     dim3(256), 0, s, p, pl.slices, part, hpart);
  return hipGetLastError();
}

}  // namespace

bool adapters_few(const AdapterProblem& p) {
  return p.M <= kMaxRows && p.places <= kMaxRows && p.R <= kMaxRank && p.K > 0 &&
         p.N <= (1 << 20);
}

size_t adapters_few_floats(const AdapterProblem& p) {
  const FewPlan pl = plan_few(p);
  return (size_t)pl.slices * ((size_t)p.M * p.N + (size_t)p.places * p.R);
}

hipError_t launch_adapters_few(const AdapterProblem& p, float* part, hipStream_t s) {
  const FewPlan pl = plan_few(p);
  return p.trans ? launch<true, 2>(p, pl, part, s) : launch<false, 4>(p, pl, part, s);
}

}  // namespace gemmf32
