// Declarations shared by the kernels around an expert layer (routing, the join
// of the experts' rows, products with 4-bit weights, the norm of many arrays) and
// their C-ABI layer.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "gemm_f32_internal.h"
#include "grouped_internal.h"

namespace gemmf32 {

// ---- routing (kernels_route.hip) ---------------------------------------------
constexpr int kMaxTop = 64;   // choices of a token: one lane each

// s = softmax or sigmoid of a token's logits; v = s + bias orders them.  Only the
// experts of the group_top best groups (by their best v, or the sum of their
// best two) can be chosen.
struct RouteProblem {
  const float* logits = nullptr;
  const float* bias = nullptr;       // NULL: none
  int64_t ldl = 0;
  int tokens = 0, experts = 0, top = 0;
  int groups = 1, group_size = 0, group_top = 1, group_best = 1;   // experts = groups group_size
  bool sigmoid = false, renorm = false;
  float scale = 1.f;
  int* choice = nullptr;             // tokens x top
  float* weight = nullptr;           // tokens x top; NULL in the gradient
  const float* dweight = nullptr;    // the gradient's: tokens x top
  float* dlogits = nullptr;
  int64_t lddl = 0;
};
hipError_t launch_route(const RouteProblem& p, hipStream_t s);
hipError_t launch_route_grad(const RouteProblem& p, hipStream_t s);

// ---- the join of the experts' rows (kernels_join.hip) --------------------------
// Entry i = t top + j counts when choice is NULL or choice[i] is in [0, groups).
struct JoinProblem {
  int64_t tokens = 0;
  int top = 0, N = 0, groups = 0;
  const int* choice = nullptr;
  const float* weight = nullptr;
  const float* H = nullptr;
  int64_t ldh = 0;
  float beta = 0.f;
  float* Y = nullptr;
  int64_t ldy = 0;
  // the gradient's
  const float* dY = nullptr;
  float* dH = nullptr;
  float* dweight = nullptr;
  int64_t lddy = 0, lddh = 0;
};
hipError_t launch_join(const JoinProblem& p, hipStream_t s);
hipError_t launch_join_grad(const JoinProblem& p, hipStream_t s);

// ---- the norm of many arrays (kernels_norm.hip) --------------------------------
// part: the workspace, norm_parts() doubles.  clip: the arrays are also scaled, into
// out (NULL: in place), where their norm is above limit.
size_t norm_parts(int64_t count, const int64_t* n);
hipError_t launch_norm(int64_t count, const float* const* x, const int64_t* n, bool clip,
                       float* const* out, float limit, float* norm, double* part, hipStream_t s);

// ---- products with 4-bit weights (kernels_q4_few.hip, kernels_q4_tiles.hip) -----
enum Q4Scale { kScaleF32 = 0, kScaleF16 = 1, kScaleBf16 = 2, kScaleE8m0 = 3 };

// The grouped product C[ic(i)] = act(alpha A[ia(i)] W_g^T + beta C[ic(i)] + bias_g) of
// GroupedProblem (places, indexes, A, C; its B is not used) with
//   W_g[n][k] = (code - zero) scale  or  e2m1(code) scale,
// two codes to a byte along k, the even k in the low half; scale and zero of
// group k >> group_shift of row n.
struct Q4Problem {
  GroupedProblem g;
  const uint8_t* codes = nullptr;
  const void* scale = nullptr;
  const uint8_t* zero = nullptr;     // NULL: 8
  int64_t ldq = 0, sq = 0;           // bytes
  int64_t lds = 0, ss = 0;           // elements
  int64_t ldz = 0, sz = 0;           // bytes
  int scale_type = kScaleF32;
  int group_shift = 5;
  bool e2m1 = false;
};
hipError_t launch_q4_few(const Q4Problem& p, const Epilogue& e, hipStream_t s);
hipError_t launch_q4_tiles(const Q4Problem& p, const Epilogue& e, hipStream_t s);

}  // namespace gemmf32
