// C ABI of the grouped products: rows ordered by group, products whose rows
// belong to different weights, the gradient of those weights, and low-rank
// adapters beside a shared projection.  Argument checks here, in the order of
// the other entry points (sizes, pitches, NULL pointers, alignment, aliasing,
// the device, reachability), then the launches: one for the rows' order and the
// products, one or two (slices and their sum) for the gradient, two for adapters
// of few rows, else three (the projection, H as a grouped product, the pass that
// adds H op(U) to Y).
#include "../../include/gemm_f32.h"

#include <hip/hip_runtime.h>

#include "gemm_f32_internal.h"
#include "grouped_internal.h"
#include "grouped_routes.h"

using gemmf32::AdapterProblem;
using gemmf32::Epilogue;
using gemmf32::GroupedProblem;

namespace {

static_assert(GEMM_F32_MAX_GROUPS == gemmf32::kMaxGroups, "one limit on groups");

constexpr int64_t kMaxElems = INT64_C(1) << 60;

// An array of a call: `count` 4-byte elements from p (0: not used).
struct Range {
  const void* p;
  int64_t count;
};

// Elements from the first to the last of `matrices` matrices of rows x cols
// (0 if they have none); -1 where that passes 2^60.
int64_t extent(int64_t rows, int64_t cols, int64_t ld, int64_t matrices = 1, int64_t stride = 0) {
  if (rows <= 0 || cols <= 0 || matrices <= 0) return 0;
  if (ld > kMaxElems / rows) return -1;
  if (matrices > 1 && stride > kMaxElems / (matrices - 1)) return -1;
  return (matrices - 1) * stride + (rows - 1) * ld + cols;
}

bool bad_dim(int64_t x) { return x < 0 || x > GEMM_F32_MAX_DIM; }
bool bad_groups(int64_t g) { return g < 0 || g > GEMM_F32_MAX_GROUPS; }
bool bad_pitch(int64_t ld, int64_t cols) { return ld < (cols > 1 ? cols : 1); }

// NULL, alignment and aliasing of the arrays: the first `written` are outputs
// and may overlap nothing.  An array that may be NULL is given with count 0
// then.
template <int N>
int check_ranges(const Range (&r)[N], int written) {
  for (const Range& x : r)
    if (x.count > 0 && !x.p) return GEMM_F32_ERR_NULL_PTR;
  for (const Range& x : r)
    if (x.count > 0 && ((uintptr_t)x.p & 3u) != 0) return GEMM_F32_ERR_POINTER;
  for (int i = 0; i < written; ++i) {
    if (r[i].count <= 0) continue;
    const uintptr_t a0 = (uintptr_t)r[i].p, a1 = a0 + (uintptr_t)r[i].count * 4;
    for (int j = 0; j < N; ++j) {
      if (j == i || r[j].count <= 0) continue;
      const uintptr_t b0 = (uintptr_t)r[j].p, b1 = b0 + (uintptr_t)r[j].count * 4;
      if (a0 < b1 && b0 < a1) return GEMM_F32_ERR_ALIAS;
    }
  }
  return GEMM_F32_OK;
}

// The device, and that it reaches every array that is used.
template <int N>
int check_reach(const Range (&r)[N], int* dev) {
  int rc = gemmf32::host_check_device(dev);
  for (int i = 0; rc == GEMM_F32_OK && i < N; ++i)
    if (r[i].count > 0) rc = gemmf32::host_check_pointer(r[i].p, *dev);
  return rc;
}

int launched(hipError_t e) {
  if (e == hipSuccess) return GEMM_F32_OK;
  (void)hipGetLastError();
  return GEMM_F32_ERR_LAUNCH;
}

template <class T>
Range used(const T* p, int64_t count) {
  return Range{p, p ? count : 0};
}

}  // namespace

extern "C" {

int gemm_f32_group_rows(int64_t n, int64_t groups, int64_t per_row, const int32_t* index,
                        int32_t* offsets, int32_t* order, int32_t* rows, void* stream) {
  if (bad_dim(n) || bad_groups(groups)) return GEMM_F32_ERR_INVALID_DIM;
  if (per_row < 1 || per_row > GEMM_F32_MAX_DIM) return GEMM_F32_ERR_INVALID_ARG;
  const Range r[] = {{offsets, groups + 1}, {order, n}, used(rows, n), {index, n}};
  int rc = check_ranges(r, 3);
  int dev = -1;
  if (rc == GEMM_F32_OK) rc = check_reach(r, &dev);
  if (rc != GEMM_F32_OK) return rc;
  return launched(gemmf32::launch_group_rows((int)n, (int)groups, (int)per_row, index, offsets,
                                             order, rows, static_cast<hipStream_t>(stream)));
}

int gemm_f32_grouped(int transB, int64_t rows, int64_t N, int64_t K, int64_t groups,
                     const int32_t* offsets, float alpha, const float* A, int64_t lda,
                     int64_t rowsA, const int32_t* indexA, const float* B, int64_t ldb,
                     int64_t strideB, float beta, float* C, int64_t ldc, int64_t rowsC,
                     const int32_t* indexC, const float* bias, int64_t strideBias,
                     int activation, void* stream) {
  const bool tb = transB != 0;
  if (bad_dim(rows) || bad_dim(N) || bad_dim(K) || bad_dim(rowsA) || bad_dim(rowsC) ||
      bad_groups(groups) || (!indexA && rowsA < rows) || (!indexC && rowsC < rows))
    return GEMM_F32_ERR_INVALID_DIM;
  const int64_t b_rows = tb ? N : K, b_cols = tb ? K : N;
  if (bad_pitch(lda, K) || bad_pitch(ldb, b_cols) || bad_pitch(ldc, N) || strideB < 0 ||
      strideBias < 0)
    return GEMM_F32_ERR_INVALID_LD;
  const bool none = rows == 0 || N == 0 || groups == 0 || rowsC == 0;
  const int64_t ea = extent(rowsA, K, lda), eb = extent(b_rows, b_cols, ldb, groups, strideB),
                ec = extent(rowsC, N, ldc), ebias = extent(1, N, N, groups, strideBias);
  if (ea < 0 || eb < 0 || ec < 0 || ebias < 0) return GEMM_F32_ERR_INVALID_LD;
  if (activation != GEMM_F32_ACT_NONE && activation != GEMM_F32_ACT_RELU)
    return GEMM_F32_ERR_INVALID_ARG;
  if (none) return GEMM_F32_OK;
  const Range r[] = {{C, ec},
                     {A, ea},
                     {B, eb},
                     {offsets, groups + 1},
                     used(indexA, rows),
                     used(indexC, rows),
                     used(bias, ebias)};
  int rc = check_ranges(r, 1);
  int dev = -1;
  if (rc == GEMM_F32_OK) rc = check_reach(r, &dev);
  if (rc != GEMM_F32_OK) return rc;
  GroupedProblem p;
  p.A = A;
  p.B = B;
  p.C = C;
  p.offsets = offsets;
  p.ia = indexA;
  p.ic = indexC;
  p.lda = lda;
  p.ldb = ldb;
  p.ldc = ldc;
  p.sb = strideB;
  p.sbias = strideBias;
  p.rows = (int)rows;
  p.groups = (int)groups;
  p.N = (int)N;
  p.K = (int)K;
  p.rows_a = (int)rowsA;
  p.rows_c = (int)rowsC;
  p.tb = tb;
  Epilogue e;
  e.alpha = alpha;
  e.beta = beta;
  e.bias = bias;
  e.act = activation;
  return launched(gemmf32::launch_grouped(p, e, static_cast<hipStream_t>(stream)));
}

int gemm_f32_grouped_wgrad(int64_t rows, int64_t M, int64_t N, int64_t groups,
                           const int32_t* offsets, float alpha, const float* A, int64_t lda,
                           int64_t rowsA, const int32_t* indexA, const float* B, int64_t ldb,
                           int64_t rowsB, const int32_t* indexB, float beta, float* C,
                           int64_t ldc, int64_t strideC, void* stream) {
  if (bad_dim(rows) || bad_dim(M) || bad_dim(N) || bad_dim(rowsA) || bad_dim(rowsB) ||
      bad_groups(groups) || (!indexA && rowsA < rows) || (!indexB && rowsB < rows))
    return GEMM_F32_ERR_INVALID_DIM;
  if (bad_pitch(lda, M) || bad_pitch(ldb, N) || bad_pitch(ldc, N) || strideC < 0)
    return GEMM_F32_ERR_INVALID_LD;
  const int64_t ea = rows > 0 ? extent(rowsA, M, lda) : 0,
                eb = rows > 0 ? extent(rowsB, N, ldb) : 0, one = extent(M, N, ldc),
                ec = extent(M, N, ldc, groups, strideC);
  if (ea < 0 || eb < 0 || one < 0 || ec < 0) return GEMM_F32_ERR_INVALID_LD;
  if (M == 0 || N == 0 || groups == 0) return GEMM_F32_OK;
  const Range r[] = {{C, ec},
                     {A, ea},
                     {B, eb},
                     {offsets, groups + 1},
                     used(indexA, rows),
                     used(indexB, rows)};
  int rc = check_ranges(r, 1);
  if (rc == GEMM_F32_OK && groups > 1 && strideC < one) rc = GEMM_F32_ERR_ALIAS;
  int dev = -1;
  if (rc == GEMM_F32_OK) rc = check_reach(r, &dev);
  if (rc != GEMM_F32_OK) return rc;
  GroupedProblem p;
  p.A = A;
  p.B = B;
  p.C = C;
  p.offsets = offsets;
  p.ia = indexA;
  p.ib = indexB;
  p.lda = lda;
  p.ldb = ldb;
  p.ldc = ldc;
  p.sc = strideC;
  p.rows = (int)rows;
  p.groups = (int)groups;
  p.M = (int)M;
  p.N = (int)N;
  p.rows_a = (int)rowsA;
  p.rows_b = (int)rowsB;
  Epilogue e;
  e.alpha = alpha;
  e.beta = beta;
  hipStream_t s = static_cast<hipStream_t>(stream);
  float* part = nullptr;
  std::unique_lock<std::mutex> turn;
  const size_t floats = gemmf32::grouped_wgrad_floats(p);
  if (floats > 0) rc = gemmf32::host_partials(dev, s, floats, &turn, &part);
  return rc != GEMM_F32_OK ? rc : launched(gemmf32::launch_grouped_wgrad(p, e, part, s));
}

int gemm_f32_adapters(int trans, int64_t M, int64_t N, int64_t K, int64_t R, int64_t groups,
                      int64_t places, const int32_t* offsets, const int32_t* order,
                      const float* scale, const float* X, int64_t ldx, const float* W,
                      int64_t ldw, const float* D, int64_t ldd, int64_t strideD, const float* U,
                      int64_t ldu, int64_t strideU, const float* bias, float* H, int64_t ldh,
                      float* Y, int64_t ldy, void* stream) {
  const bool t = trans != 0;
  if (bad_dim(M) || bad_dim(N) || bad_dim(K) || bad_dim(R) || bad_dim(places) ||
      bad_groups(groups))
    return GEMM_F32_ERR_INVALID_DIM;
  const int64_t w_rows = t ? N : K, w_cols = t ? K : N, d_rows = t ? R : K, d_cols = t ? K : R,
                u_rows = t ? N : R, u_cols = t ? R : N;
  if (bad_pitch(ldx, K) || bad_pitch(ldw, w_cols) || bad_pitch(ldy, N)) return GEMM_F32_ERR_INVALID_LD;
  const bool some = R > 0 && groups > 0 && places > 0;
  if (some && (bad_pitch(ldd, d_cols) || bad_pitch(ldu, u_cols) || bad_pitch(ldh, R) ||
               strideD < 0 || strideU < 0))
    return GEMM_F32_ERR_INVALID_LD;
  const int64_t ex = extent(M, K, ldx), ew = extent(w_rows, w_cols, ldw), ey = extent(M, N, ldy);
  const int64_t ed = some ? extent(d_rows, d_cols, ldd, groups, strideD) : 0,
                eu = some ? extent(u_rows, u_cols, ldu, groups, strideU) : 0,
                eh = some ? extent(places, R, ldh) : 0;
  if (ex < 0 || ew < 0 || ey < 0 || ed < 0 || eu < 0 || eh < 0) return GEMM_F32_ERR_INVALID_LD;
  if (M == 0 || N == 0) return GEMM_F32_OK;
  const Range r[] = {{Y, ey},
                     {H, eh},
                     {X, ex},
                     {W, ew},
                     {D, ed},
                     {U, eu},
                     {offsets, some ? groups + 1 : 0},
                     {order, some ? places : 0},
                     used(scale, some ? groups : 0),
                     used(bias, N)};
  int rc = check_ranges(r, 2);
  int dev = -1;
  if (rc == GEMM_F32_OK) rc = check_reach(r, &dev);
  if (rc != GEMM_F32_OK) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (!some)
    return gemm_f32_fused(0, trans, M, N, K, 1.f, X, ldx, W, ldw, 0.f, Y, ldy, bias,
                          GEMM_F32_ACT_NONE, stream);
  AdapterProblem a{};
  a.X = X;
  a.W = W;
  a.D = D;
  a.U = U;
  a.scale = scale;
  a.bias = bias;
  a.offsets = offsets;
  a.order = order;
  a.H = H;
  a.Y = Y;
  a.ldx = ldx;
  a.ldw = ldw;
  a.ldd = ldd;
  a.sd = strideD;
  a.ldu = ldu;
  a.su = strideU;
  a.ldh = ldh;
  a.ldy = ldy;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.R = (int)R;
  a.groups = (int)groups;
  a.places = (int)places;
  a.trans = t;
  if (gemmf32::adapters_few(a)) {
    float* part = nullptr;
    std::unique_lock<std::mutex> turn;
    rc = gemmf32::host_partials(dev, s, gemmf32::adapters_few_floats(a), &turn, &part);
    return rc != GEMM_F32_OK ? rc : launched(gemmf32::launch_adapters_few(a, part, s));
  }
  GroupedProblem b;   // the projection, all rows in one group
  b.A = X;
  b.lda = ldx;
  b.rows_a = b.rows_c = b.rows = (int)M;
  b.B = W;
  b.ldb = ldw;
  b.C = Y;
  b.ldc = ldy;
  b.groups = 1;
  b.N = (int)N;
  b.K = (int)K;
  b.tb = t;
  if (gemmf32::projection_grouped(b)) {
    Epilogue e;
    e.bias = bias;
    rc = launched(gemmf32::launch_grouped(b, e, s));
  } else {
    rc = gemm_f32_fused(0, trans, M, N, K, 1.f, X, ldx, W, ldw, 0.f, Y, ldy, bias,
                        GEMM_F32_ACT_NONE, stream);
  }
  if (rc != GEMM_F32_OK) return rc;
  GroupedProblem p;   // H = s_g X[order] op(D_g)
  p.A = X;
  p.lda = ldx;
  p.rows_a = (int)M;
  p.ia = order;
  p.B = D;
  p.ldb = ldd;
  p.sb = strideD;
  p.C = H;
  p.ldc = ldh;
  p.rows_c = (int)places;
  p.offsets = offsets;
  p.gscale = scale;
  p.rows = (int)places;
  p.groups = (int)groups;
  p.N = (int)R;
  p.K = (int)K;
  p.tb = t;
  rc = launched(gemmf32::launch_grouped(p, Epilogue{}, s));
  return rc != GEMM_F32_OK ? rc : launched(gemmf32::launch_adapters_add(a, s));
}

}  // extern "C"
