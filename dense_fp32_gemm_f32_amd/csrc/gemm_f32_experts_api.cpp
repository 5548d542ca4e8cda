// C ABI of the operators around an expert layer: routing and its gradient, the
// join of the experts' rows and its gradient, products with 4-bit weights, the norm
// of many arrays and clipping.  Argument checks here, in the order of the other
// entry points, then the launches.
#include "../../include/gemm_f32.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "experts_internal.h"
#include "host_checks.h"
#include "q4_routes.h"

using gemmf32::Epilogue;
using gemmf32::JoinProblem;
using gemmf32::Q4Problem;
using gemmf32::RouteProblem;
using namespace gemmf32::checks;

namespace {

static_assert(GEMM_F32_MAX_TOP == gemmf32::kMaxTop, "one limit on a token's choices");
static_assert(GEMM_F32_SCALE_E8M0 == gemmf32::kScaleE8m0, "one numbering of the scales' types");

constexpr int64_t kMaxArrays = INT64_C(1) << 20, kMaxArray = INT64_C(1) << 40;

bool bad_route(int64_t tokens, int64_t experts, int64_t top) {
  return bad_dim(tokens) || bad_groups(experts) || top < 0 || top > GEMM_F32_MAX_TOP;
}
bool bad_score(int score) {
  return score != GEMM_F32_SCORE_SOFTMAX && score != GEMM_F32_SCORE_SIGMOID;
}

// The arrays of a norm; `out` NULL for the norm alone.
struct Arrays {
  int64_t count;
  const float* const* x;
  const int64_t* n;
  float* const* out;
  const float* y(int64_t i) const { return out ? out[i] : x[i]; }
};

// One array's bytes [from, to).
struct Span {
  uintptr_t from, to;
  bool writes;
};

// Do two of the spans overlap, one of which is written?
bool overlaps(std::vector<Span>& v) {
  std::sort(v.begin(), v.end(),
            [](const Span& a, const Span& b) { return a.from < b.from; });
  // how far those before it reach that are read, and that are written
  uintptr_t read_to = 0, write_to = 0;
  for (const Span& s : v) {
    if (s.from < write_to || (s.writes && s.from < read_to)) return true;
    if (s.writes)
      write_to = std::max(write_to, s.to);
    else
      read_to = std::max(read_to, s.to);
  }
  return false;
}

int check_arrays(const Arrays& a, const float* norm, bool clip, int* dev) {
  if (a.count < 0 || a.count > kMaxArrays) return GEMM_F32_ERR_INVALID_DIM;
  if (a.count > 0 && (!a.x || !a.n)) return GEMM_F32_ERR_NULL_PTR;
  for (int64_t i = 0; i < a.count; ++i)
    if (a.n[i] < 0 || a.n[i] > kMaxArray) return GEMM_F32_ERR_INVALID_DIM;
  if (!norm) return GEMM_F32_ERR_NULL_PTR;
  for (int64_t i = 0; i < a.count; ++i)
    if (a.n[i] > 0 && (!a.x[i] || (clip && !a.y(i)))) return GEMM_F32_ERR_NULL_PTR;
  auto odd = [](const float* p) { return ((uintptr_t)p & 3u) != 0; };
  if (odd(norm)) return GEMM_F32_ERR_POINTER;
  for (int64_t i = 0; i < a.count; ++i)
    if (a.n[i] > 0 && (odd(a.x[i]) || (clip && odd(a.y(i))))) return GEMM_F32_ERR_POINTER;
  std::vector<Span> spans;
  spans.reserve((size_t)(a.count * 2 + 1));
  auto span = [&](const float* p, int64_t n, bool writes) {
    spans.push_back(Span{(uintptr_t)p, (uintptr_t)p + (uintptr_t)n * 4, writes});
  };
  span(norm, 1, true);
  for (int64_t i = 0; i < a.count; ++i) {
    if (a.n[i] <= 0) continue;
    const bool in_place = clip && a.y(i) == a.x[i];
    if (!in_place) span(a.x[i], a.n[i], false);
    if (clip) span(a.y(i), a.n[i], true);
  }
  if (overlaps(spans)) return GEMM_F32_ERR_ALIAS;
  int rc = gemmf32::host_check_device(dev);
  if (rc == GEMM_F32_OK) rc = gemmf32::host_check_pointer(norm, *dev);
  for (int64_t i = 0; rc == GEMM_F32_OK && i < a.count; ++i) {
    if (a.n[i] <= 0) continue;
    rc = gemmf32::host_check_pointer(a.x[i], *dev);
    if (rc == GEMM_F32_OK && clip && a.y(i) != a.x[i])
      rc = gemmf32::host_check_pointer(a.y(i), *dev);
  }
  return rc;
}

int run_norm(const Arrays& a, float limit, float* norm, bool clip, void* stream) {
  int dev = -1, rc;
  try {
    rc = check_arrays(a, norm, clip, &dev);
  } catch (const std::bad_alloc&) {
    return GEMM_F32_ERR_WORKSPACE;
  }
  if (rc != GEMM_F32_OK) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  float* part = nullptr;
  std::unique_lock<std::mutex> turn;
  const size_t parts = gemmf32::norm_parts(a.count, a.n);
  if (parts > 0) rc = gemmf32::host_partials(dev, s, 2 * parts, &turn, &part);
  if (rc != GEMM_F32_OK) return rc;
  return launched(gemmf32::launch_norm(a.count, a.x, a.n, clip, a.out, limit, norm,
                                       reinterpret_cast<double*>(part), s));
}

// Both entry points of the 4-bit products: without offsets, one group of all rows.
int run_q4(int64_t rows, int64_t N, int64_t K, int64_t groups, const int32_t* offsets, float alpha,
           const float* A, int64_t lda, int64_t rowsA, const int32_t* indexA, int format,
           int64_t group, const uint8_t* codes, int64_t ldq, int64_t strideQ, int scale_type,
           const void* scale, int64_t lds, int64_t strideS, const uint8_t* zero, int64_t ldz,
           int64_t strideZ, float beta, float* C, int64_t ldc, int64_t rowsC,
           const int32_t* indexC, const float* bias, int64_t strideBias, int activation,
           bool grouped, void* stream) {
  if (bad_dim(rows) || bad_dim(N) || bad_dim(K) || bad_dim(rowsA) || bad_dim(rowsC) ||
      bad_groups(groups) || (!indexA && rowsA < rows) || (!indexC && rowsC < rows))
    return GEMM_F32_ERR_INVALID_DIM;
  if (group < 32 || (group & (group - 1)) != 0) return GEMM_F32_ERR_INVALID_ARG;
  const int64_t bytes = (K + 1) / 2, along = K > 0 ? (K - 1) / group + 1 : 0;
  if (bad_pitch(lda, K) || bad_pitch(ldq, bytes) || bad_pitch(lds, along) ||
      (zero && bad_pitch(ldz, along)) || bad_pitch(ldc, N) || strideQ < 0 || strideS < 0 ||
      (zero && strideZ < 0) || strideBias < 0)
    return GEMM_F32_ERR_INVALID_LD;
  const int64_t ea = extent(rowsA, K, lda), eq = extent(N, bytes, ldq, groups, strideQ),
                es = extent(N, along, lds, groups, strideS),
                ez = zero ? extent(N, along, ldz, groups, strideZ) : 0,
                ec = extent(rowsC, N, ldc), ebias = extent(1, N, N, groups, strideBias);
  if (ea < 0 || eq < 0 || es < 0 || ez < 0 || ec < 0 || ebias < 0) return GEMM_F32_ERR_INVALID_LD;
  const bool e2m1 = format == GEMM_F32_Q4_E2M1;
  if ((format != GEMM_F32_Q4_INT && !e2m1) || (e2m1 && zero) || scale_type < GEMM_F32_SCALE_F32 ||
      scale_type > GEMM_F32_SCALE_E8M0 ||
      (activation != GEMM_F32_ACT_NONE && activation != GEMM_F32_ACT_RELU))
    return GEMM_F32_ERR_INVALID_ARG;
  if (rows == 0 || N == 0 || groups == 0 || rowsC == 0) return GEMM_F32_OK;
  static const int kScaleBytes[] = {4, 2, 2, 1};
  const Range r[] = {{C, ec},
                     {A, ea},
                     {codes, eq, 1},
                     {scale, es, kScaleBytes[scale_type]},
                     used(zero, ez),
                     {offsets, grouped ? groups + 1 : 0},
                     used(indexA, rows),
                     used(indexC, rows),
                     used(bias, ebias)};
  int rc = check_ranges(r, 1);
  int dev = -1;
  if (rc == GEMM_F32_OK) rc = check_reach(r, &dev);
  if (rc != GEMM_F32_OK) return rc;
  Q4Problem p;
  p.g.A = A;
  p.g.lda = lda;
  p.g.rows_a = (int)rowsA;
  p.g.ia = indexA;
  p.g.C = C;
  p.g.ldc = ldc;
  p.g.rows_c = (int)rowsC;
  p.g.ic = indexC;
  p.g.offsets = offsets;
  p.g.rows = (int)rows;
  p.g.groups = (int)groups;
  p.g.N = (int)N;
  p.g.K = (int)K;
  p.g.sbias = strideBias;
  p.codes = codes;
  p.ldq = ldq;
  p.sq = strideQ;
  p.scale = scale;
  p.scale_type = scale_type;
  p.lds = lds;
  p.ss = strideS;
  p.zero = zero;
  p.ldz = ldz;
  p.sz = strideZ;
  p.e2m1 = e2m1;
  // a group beyond K holds every k: a shift of 31 does as well
  while ((INT64_C(1) << p.group_shift) < group && p.group_shift < 31) ++p.group_shift;
  Epilogue e;
  e.alpha = alpha;
  e.beta = beta;
  e.bias = bias;
  e.act = activation;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return launched(gemmf32::q4_few(p) ? gemmf32::launch_q4_few(p, e, s)
                                     : gemmf32::launch_q4_tiles(p, e, s));
}

}  // namespace

extern "C" {

int gemm_f32_route(int64_t tokens, int64_t experts, int64_t top, const float* logits,
                   int64_t ldl, const float* bias, int score, int64_t groups, int64_t group_top,
                   int group_best, int renorm, float scale, int32_t* choice, float* weight,
                   void* stream) {
  if (bad_route(tokens, experts, top) || groups < 1 || groups > GEMM_F32_MAX_GROUPS ||
      experts % groups != 0)
    return GEMM_F32_ERR_INVALID_DIM;
  if (bad_pitch(ldl, experts)) return GEMM_F32_ERR_INVALID_LD;
  const int64_t el = extent(tokens, experts, ldl);
  if (el < 0) return GEMM_F32_ERR_INVALID_LD;
  if (bad_score(score) || group_top < 1 || group_top > groups ||
      (group_best != 1 && group_best != 2))
    return GEMM_F32_ERR_INVALID_ARG;
  if (tokens == 0 || top == 0) return GEMM_F32_OK;
  const Range r[] = {{choice, tokens * top},
                     {weight, tokens * top},
                     {logits, el},
                     used(bias, experts)};
  int rc = check_ranges(r, 2);
  int dev = -1;
  if (rc == GEMM_F32_OK) rc = check_reach(r, &dev);
  if (rc != GEMM_F32_OK) return rc;
  RouteProblem p;
  p.logits = logits;
  p.bias = bias;
  p.ldl = ldl;
  p.tokens = (int)tokens;
  p.experts = (int)experts;
  p.top = (int)top;
  p.groups = (int)groups;
  p.group_size = (int)(experts / groups);
  p.group_top = (int)group_top;
  p.group_best = group_best;
  p.sigmoid = score == GEMM_F32_SCORE_SIGMOID;
  p.renorm = renorm != 0;
  p.scale = scale;
  p.choice = choice;
  p.weight = weight;
  return launched(gemmf32::launch_route(p, static_cast<hipStream_t>(stream)));
}

int gemm_f32_route_grad(int64_t tokens, int64_t experts, int64_t top, const float* logits,
                        int64_t ldl, int score, int renorm, float scale, const int32_t* choice,
                        const float* dweight, float* dlogits, int64_t lddl, void* stream) {
  if (bad_route(tokens, experts, top)) return GEMM_F32_ERR_INVALID_DIM;
  if (bad_pitch(ldl, experts) || bad_pitch(lddl, experts)) return GEMM_F32_ERR_INVALID_LD;
  const int64_t el = extent(tokens, experts, ldl), ed = extent(tokens, experts, lddl);
  if (el < 0 || ed < 0) return GEMM_F32_ERR_INVALID_LD;
  if (bad_score(score)) return GEMM_F32_ERR_INVALID_ARG;
  if (tokens == 0 || experts == 0) return GEMM_F32_OK;
  const Range r[] = {{dlogits, ed}, {logits, el}, {choice, tokens * top}, {dweight, tokens * top}};
  int rc = check_ranges(r, 1);
  int dev = -1;
  if (rc == GEMM_F32_OK) rc = check_reach(r, &dev);
  if (rc != GEMM_F32_OK) return rc;
  RouteProblem p;
  p.logits = logits;
  p.ldl = ldl;
  p.tokens = (int)tokens;
  p.experts = (int)experts;
  p.top = (int)top;
  p.sigmoid = score == GEMM_F32_SCORE_SIGMOID;
  p.renorm = renorm != 0;
  p.scale = scale;
  p.choice = const_cast<int32_t*>(choice);
  p.dweight = dweight;
  p.dlogits = dlogits;
  p.lddl = lddl;
  return launched(gemmf32::launch_route_grad(p, static_cast<hipStream_t>(stream)));
}

int gemm_f32_join_rows(int64_t tokens, int64_t top, int64_t N, const float* H, int64_t ldh,
                       const float* weight, const int32_t* choice, int64_t groups, float beta,
                       float* Y, int64_t ldy, void* stream) {
  if (bad_dim(tokens) || bad_dim(top) || bad_dim(N) || bad_groups(groups) ||
      (top > 0 && tokens > GEMM_F32_MAX_DIM / top))
    return GEMM_F32_ERR_INVALID_DIM;
  if (bad_pitch(ldh, N) || bad_pitch(ldy, N)) return GEMM_F32_ERR_INVALID_LD;
  const int64_t entries = tokens * top, eh = extent(entries, N, ldh), ey = extent(tokens, N, ldy);
  if (eh < 0 || ey < 0) return GEMM_F32_ERR_INVALID_LD;
  if (tokens == 0 || N == 0) return GEMM_F32_OK;
  const Range r[] = {{Y, ey}, {H, eh}, {weight, entries}, used(choice, entries)};
  int rc = check_ranges(r, 1);
  int dev = -1;
  if (rc == GEMM_F32_OK) rc = check_reach(r, &dev);
  if (rc != GEMM_F32_OK) return rc;
  JoinProblem p;
  p.tokens = tokens;
  p.top = (int)top;
  p.N = (int)N;
  p.groups = (int)groups;
  p.choice = choice;
  p.weight = weight;
  p.H = H;
  p.ldh = ldh;
  p.beta = beta;
  p.Y = Y;
  p.ldy = ldy;
  return launched(gemmf32::launch_join(p, static_cast<hipStream_t>(stream)));
}

int gemm_f32_join_rows_grad(int64_t tokens, int64_t top, int64_t N, const float* dY, int64_t lddy,
                            const float* H, int64_t ldh, const float* weight,
                            const int32_t* choice, int64_t groups, float* dH, int64_t lddh,
                            float* dweight, void* stream) {
  if (bad_dim(tokens) || bad_dim(top) || bad_dim(N) || bad_groups(groups) ||
      (top > 0 && tokens > GEMM_F32_MAX_DIM / top))
    return GEMM_F32_ERR_INVALID_DIM;
  if (bad_pitch(lddy, N) || bad_pitch(ldh, N) || bad_pitch(lddh, N))
    return GEMM_F32_ERR_INVALID_LD;
  const int64_t entries = tokens * top, eh = extent(entries, N, ldh),
                ed = extent(entries, N, lddh), ey = extent(tokens, N, lddy);
  if (eh < 0 || ed < 0 || ey < 0) return GEMM_F32_ERR_INVALID_LD;
  if (entries == 0) return GEMM_F32_OK;
  const Range r[] = {{dH, ed},          {dweight, entries},      {dY, ey}, {H, eh},
                     {weight, entries}, used(choice, entries)};
  int rc = check_ranges(r, 2);
  int dev = -1;
  if (rc == GEMM_F32_OK) rc = check_reach(r, &dev);
  if (rc != GEMM_F32_OK) return rc;
  JoinProblem p;
  p.tokens = tokens;
  p.top = (int)top;
  p.N = (int)N;
  p.groups = (int)groups;
  p.choice = choice;
  p.weight = weight;
  p.H = H;
  p.ldh = ldh;
  p.dY = dY;
  p.lddy = lddy;
  p.dH = dH;
  p.lddh = lddh;
  p.dweight = dweight;
  return launched(gemmf32::launch_join_grad(p, static_cast<hipStream_t>(stream)));
}

int gemm_f32_q4_grouped(int64_t rows, int64_t N, int64_t K, int64_t groups,
                        const int32_t* offsets, float alpha, const float* A, int64_t lda,
                        int64_t rowsA, const int32_t* indexA, int format, int64_t group,
                        const uint8_t* codes, int64_t ldq, int64_t strideQ, int scale_type,
                        const void* scale, int64_t lds, int64_t strideS, const uint8_t* zero,
                        int64_t ldz, int64_t strideZ, float beta, float* C, int64_t ldc,
                        int64_t rowsC, const int32_t* indexC, const float* bias,
                        int64_t strideBias, int activation, void* stream) {
  return run_q4(rows, N, K, groups, offsets, alpha, A, lda, rowsA, indexA, format,
                         group, codes, ldq, strideQ, scale_type, scale, lds, strideS, zero, ldz,
                         strideZ, beta, C, ldc, rowsC, indexC, bias, strideBias, activation,
                true, stream);
}

int gemm_f32_q4(int64_t M, int64_t N, int64_t K, float alpha, const float* A, int64_t lda,
                int format, int64_t group, const uint8_t* codes, int64_t ldq, int scale_type,
                const void* scale, int64_t lds, const uint8_t* zero, int64_t ldz, float beta,
                float* C, int64_t ldc, const float* bias, int activation, void* stream) {
  return run_q4(M, N, K, 1, nullptr, alpha, A, lda, M, nullptr, format, group,
                         codes, ldq, 0, scale_type, scale, lds, 0, zero, ldz, 0, beta, C, ldc, M,
                         nullptr, bias, 0, activation, false, stream);
}

int gemm_f32_norm(int64_t count, const float* const* x, const int64_t* n, float* norm,
                  void* stream) {
  return run_norm(Arrays{count, x, n, nullptr}, 0.f, norm, false, stream);
}

int gemm_f32_clip(int64_t count, const float* const* x, const int64_t* n, float* const* out,
                  float max_norm, float* norm, void* stream) {
  if (count < 0 || count > kMaxArrays) return GEMM_F32_ERR_INVALID_DIM;
  if (!(max_norm >= 0.f)) return GEMM_F32_ERR_INVALID_ARG;
  return run_norm(Arrays{count, x, n, out}, max_norm, norm, true, stream);
}

}  // extern "C"
