// Declarations shared by the grouped products' kernels and their C-ABI layer:
// products whose rows (or, for the weights' gradient, whose K) are split over
// groups by offsets that only the device knows.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <mutex>

#include "gemm_f32_internal.h"

namespace gemmf32 {

// The host checks and the per-stream partial sums that gemm_f32_api.cpp has.
int host_check_device(int* dev);                    // gfx950 only; the current device
int host_check_pointer(const void* p, int dev);     // memory that device can reach
// turn: keeps other host threads' calls on this stream from launching until the
// caller lets it go, behind its last launch that uses the partial sums
int host_partials(int dev, hipStream_t s, size_t floats, std::unique_lock<std::mutex>* turn,
                  float** out);

// Place i (0 <= i < rows) belongs to group g when offsets[g] <= i < offsets[g+1].
// Product (launch_grouped):   C[ic(i)] = act(alpha s_g A[ia(i)] op(B_g) + beta C[ic(i)] + bias_g)
// Gradient (launch_grouped_wgrad): C_g = alpha sum_i A[ia(i)]^T B[ib(i)] + beta C_g
// Without offsets (product only) all places are of group 0.
// An index array that is NULL is the identity.  s_g = gscale[g], 1 when NULL.
struct GroupedProblem {
  const float* A = nullptr;
  const float* B = nullptr;
  float* C = nullptr;
  const int* offsets = nullptr;
  const int* ia = nullptr;
  const int* ib = nullptr;   // gradient only
  const int* ic = nullptr;   // product only
  const float* gscale = nullptr;
  int64_t lda = 0, ldb = 0, ldc = 0;
  int64_t sb = 0, sc = 0, sbias = 0;   // strides of B_g, C_g and bias_g
  int rows = 0, groups = 0;
  int M = 0, N = 0, K = 0;             // M: gradient only; K: product only
  int rows_a = 0, rows_b = 0, rows_c = 0;
  bool tb = false;                     // product: B_g stored N x K
};

hipError_t launch_grouped(const GroupedProblem& p, const Epilogue& e, hipStream_t s);
// the same for few rows in a group, or few columns (kernels_grouped_rows.hip)
hipError_t launch_grouped_rows(const GroupedProblem& p, const Epilogue& e, hipStream_t s);
// The gradient, and the floats of workspace (part) it takes.
hipError_t launch_grouped_wgrad(const GroupedProblem& p, const Epilogue& e, float* part,
                                hipStream_t s);
size_t grouped_wgrad_floats(const GroupedProblem& p);
// the same for M or N of at most 64 (kernels_grouped_wgrad_thin.hip), and the
// launch that adds the slices' sums in part, slices x groups x M x N
size_t wgrad_thin_floats(const GroupedProblem& p);
hipError_t launch_wgrad_thin(const GroupedProblem& p, const Epilogue& e, float* part,
                             hipStream_t s);
hipError_t launch_wgrad_join(const GroupedProblem& p, const Epilogue& e, int slices,
                             const float* part, hipStream_t s);

// gemm_f32_adapters after its checks: matrices as stored (trans: each transposed).
struct AdapterProblem {
  const float *X, *W, *D, *U, *scale, *bias;
  const int *offsets, *order;
  float *H, *Y;
  int64_t ldx, ldw, ldd, sd, ldu, su, ldh, ldy;
  int M, N, K, R, groups, places;
  bool trans;
};
// Y[order[i]] += H[i] op(U_g) (kernels_adapters.hip)
hipError_t launch_adapters_add(const AdapterProblem& p, hipStream_t s);
// few rows: one launch of partial sums and one that joins them
// (kernels_adapters_few.hip); the floats of workspace it takes
bool adapters_few(const AdapterProblem& p);
size_t adapters_few_floats(const AdapterProblem& p);
hipError_t launch_adapters_few(const AdapterProblem& p, float* part, hipStream_t s);

// offsets, order and rows (may be NULL) of gemm_f32_group_rows
hipError_t launch_group_rows(int n, int groups, int per_row, const int* index, int* offsets,
                             int* order, int* rows, hipStream_t s);

constexpr int kMaxGroups = 1024;

// A grid of n workgroups (n below 2^31): the launch takes fewer than 2^32
// threads along x, so larger grids go on along y.  tile_id() numbers them.
constexpr int64_t kGridX = 1 << 21;
inline dim3 tile_grid(int64_t n) {
  const int64_t x = n < kGridX ? n : kGridX;
  return dim3((unsigned)x, (unsigned)((n + x - 1) / x));
}

#if defined(__HIP__)
constexpr unsigned kXcds = 8;
__device__ __forceinline__ unsigned tile_id() { return blockIdx.y * gridDim.x + blockIdx.x; }

// Position `at` of n positions dealt to the XCDs round robin by workgroup id, so
// that each XCD has a contiguous range; -1 past the end.
__device__ __forceinline__ int xcd_position(unsigned at, unsigned n) {
  const unsigned x = at % kXcds, q = n / kXcds, rem = n % kXcds;
  if (at / kXcds >= q + (x < rem ? 1u : 0u)) return -1;
  return (int)(x * q + min(x, rem) + at / kXcds);
}

// Group g's places, taken into [0, rows]; a group that ends before it begins
// is empty.  Without offsets there is one group, of all places.
__device__ __forceinline__ void group_span(const int* offsets, int g, int rows, int& begin,
                                           int& end) {
  begin = offsets ? min(max(offsets[g], 0), rows) : 0;
  end = offsets ? max(begin, min(offsets[g + 1], rows)) : rows;
}

// Inclusive sum over the lanes of a wave, held below `cap`.
__device__ __forceinline__ unsigned wave_scan(unsigned x, unsigned cap, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const unsigned y = __shfl_up(x, d);
    if (lane >= d) x = min(x + y, cap);
  }
  return x;
}

// The row tiles of all groups in order, bm places each (a group's last one
// part full), as tile numbers 0 .. total - 1.  Each wave computes it alone from
// the offsets: one load of 64 groups, a scan, a ballot.
//   total()   the number of row tiles, held below cap
//   find(t)   the group of row tile t < total(): its number, its places, and
//             the first of its row tiles
struct RowTiles {
  const int* offsets;
  int groups, rows, bm, lane;
  unsigned cap;
  unsigned first_incl;   // the scan of groups 0 .. 63, kept for find

  __device__ __forceinline__ unsigned scan_at(int base) const {
    unsigned x = 0;
    if (base + lane < groups) {
      int b, e;
      group_span(offsets, base + lane, rows, b, e);
      x = (unsigned)((e - b + bm - 1) / bm);
    }
    return wave_scan(x, cap, lane);
  }
  __device__ __forceinline__ unsigned total() {
    unsigned sum = 0;
    for (int base = 0; base < groups; base += 64) {
      const unsigned incl = scan_at(base);
      if (base == 0) first_incl = incl;
      sum = min(sum + (unsigned)__builtin_amdgcn_readlane(incl, 63), cap);
    }
    return sum;
  }
  __device__ __forceinline__ bool find(unsigned t, int& g, int& begin, int& end,
                                       unsigned& first) const {
    unsigned sum = 0;
    for (int base = 0; base < groups; base += 64) {
      const unsigned incl = base == 0 ? first_incl : scan_at(base);
      const unsigned long long past = __ballot(sum + incl > t);
      if (past) {
        const int l = __builtin_ctzll(past);
        const unsigned before = l > 0 ? (unsigned)__builtin_amdgcn_readlane(incl, l - 1) : 0u;
        g = base + l;
        first = sum + before;
        group_span(offsets, g, rows, begin, end);
        begin = __builtin_amdgcn_readfirstlane(begin);
        end = __builtin_amdgcn_readfirstlane(end);
        return true;
      }
      sum = min(sum + (unsigned)__builtin_amdgcn_readlane(incl, 63), cap);
    }
    return false;
  }
};
#endif

// Most row tiles of bm places that `rows` places in `groups` groups can need.
inline int64_t most_row_tiles(int64_t rows, int64_t groups, int bm) {
  return rows / bm + (groups < rows ? groups : rows);
}

}  // namespace gemmf32
