// Argument checks shared by the C-ABI layers of the grouped products and of the
// operators around an expert layer.  Host code only.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/gemm_f32.h"
#include "grouped_internal.h"

namespace gemmf32 {
namespace checks {

constexpr int64_t kMaxElems = INT64_C(1) << 60;

// An array of a call: `count` elements of `size` bytes from p (0: not used).
struct Range {
  const void* p;
  int64_t count;
  int size = 4;
};

// Elements from the first to the last of `matrices` matrices of rows x cols
// (0 if they have none); -1 where that passes 2^60.
inline int64_t extent(int64_t rows, int64_t cols, int64_t ld, int64_t matrices = 1,
                      int64_t stride = 0) {
  if (rows <= 0 || cols <= 0 || matrices <= 0) return 0;
  if (ld > kMaxElems / rows) return -1;
  if (matrices > 1 && stride > kMaxElems / (matrices - 1)) return -1;
  return (matrices - 1) * stride + (rows - 1) * ld + cols;
}

inline bool bad_dim(int64_t x) { return x < 0 || x > GEMM_F32_MAX_DIM; }
inline bool bad_groups(int64_t g) { return g < 0 || g > GEMM_F32_MAX_GROUPS; }
inline bool bad_pitch(int64_t ld, int64_t cols) { return ld < (cols > 1 ? cols : 1); }

// NULL, alignment (each element's own) and aliasing of the arrays: the first
// `written` are outputs and may overlap nothing.  An array that may be NULL is
// given with count 0 then.
template <int N>
int check_ranges(const Range (&r)[N], int written) {
  for (const Range& x : r)
    if (x.count > 0 && !x.p) return GEMM_F32_ERR_NULL_PTR;
  for (const Range& x : r)
    if (x.count > 0 && (uintptr_t)x.p % (unsigned)x.size != 0) return GEMM_F32_ERR_POINTER;
  for (int i = 0; i < written; ++i) {
    if (r[i].count <= 0) continue;
    const uintptr_t a0 = (uintptr_t)r[i].p, a1 = a0 + (uintptr_t)r[i].count * r[i].size;
    for (int j = 0; j < N; ++j) {
      if (j == i || r[j].count <= 0) continue;
      const uintptr_t b0 = (uintptr_t)r[j].p, b1 = b0 + (uintptr_t)r[j].count * r[j].size;
      if (a0 < b1 && b0 < a1) return GEMM_F32_ERR_ALIAS;
    }
  }
  return GEMM_F32_OK;
}

// The device, and that it reaches every array that is used.
template <int N>
int check_reach(const Range (&r)[N], int* dev) {
  int rc = host_check_device(dev);
  for (int i = 0; rc == GEMM_F32_OK && i < N; ++i)
    if (r[i].count > 0) rc = host_check_pointer(r[i].p, *dev);
  return rc;
}

inline int launched(hipError_t e) {
  if (e == hipSuccess) return GEMM_F32_OK;
  (void)hipGetLastError();
  return GEMM_F32_ERR_LAUNCH;
}

template <class T>
Range used(const T* p, int64_t count) {
  return Range{p, p ? count : 0, (int)sizeof(T)};
}

}  // namespace checks
}  // namespace gemmf32
