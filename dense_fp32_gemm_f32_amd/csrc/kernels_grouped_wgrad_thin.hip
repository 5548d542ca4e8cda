// The gradient of grouped weights with few rows or few columns, such as a low-rank
// factor's or a bias's (gfx950): for every group g, over its places i, C_g = alpha
// sum_i A[ia(i)]^T B[ib(i)] + beta C_g, where M or N is at most 64.
//
// Bound by reading the wide operand once.  A workgroup owns 64 columns of the
// wide operand by 16 NB of the thin one; its 8 waves take the places 64 at a
// time, in turn.  With v_mfma_f32_16x16x4_f32 lane (h = l / 16, c = l % 16) holds the
// wide columns 4 c + j (one 16-byte load, j = 0 .. 3) and the thin columns NB c + j of
// place 4 s + h in step s, so every load reads whole runs of a row; the index
// entries of 64 places are loaded together and handed around.  The waves' sums are
// added in LDS in wave order.  Long groups are cut into slices, one workgroup
// each, whose sums go through a workspace and a second launch.
#include <algorithm>

#include "grouped_internal.h"
#include "mfma_common.h"

namespace gemmf32 {
namespace {

using namespace mfma;

typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8, kWide = 64;
constexpr int kMaxSlices = 32;
static __device__ __attribute__((aligned(16))) const float kZeroChunk[4] = {0.f, 0.f, 0.f, 0.f};

// One operand: its matrix and the rows its places name.
struct Rows {
  const float* X;
  int64_t ld;
  const int* index;
  int limit, cols;
};

// kWideA: the wide operand is A (M wide), else B.
template <int NB, bool kWideA>
__global__ void __launch_bounds__(kWaves * 64)
    wgrad_thin_kernel(GroupedProblem p, Epilogue ep, int tiles, int strips, int slices,
                      float* part) {
  constexpr int kThin = 16 * NB;
  __shared__ float red[kWaves * kWide * kThin];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 4, c = lane & 15;
  // id -> (group, slice, strip, wide tile)
  unsigned id = tile_id();
  const int tile = (int)(id % tiles);
  id /= tiles;
  const int strip = (int)(id % strips);
  id /= strips;
  const int slice = (int)(id % slices), g = (int)(id / slices);
  if (g >= p.groups) return;
  int begin, end;
  group_span(p.offsets, g, p.rows, begin, end);
  // this slice's places: whole turns of the waves
  const int64_t turn = 64 * kWaves;
  const int64_t len = ((int64_t)(end - begin) + slices * turn - 1) / (slices * turn) * turn;
  const int s0 = (int)min((int64_t)end, begin + slice * len), s1 = (int)min((int64_t)end, s0 + len);

  const Rows wide = kWideA ? Rows{p.A, p.lda, p.ia, p.rows_a, p.M} : Rows{p.B, p.ldb, p.ib, p.rows_b, p.N};
  const Rows thin = kWideA ? Rows{p.B, p.ldb, p.ib, p.rows_b, p.N} : Rows{p.A, p.lda, p.ia, p.rows_a, p.M};
  const int w0 = tile * kWide, t0 = strip * kThin;
  // of this lane's columns, those inside
  const int w_in = max(0, min(4, wide.cols - w0 - 4 * c));
  const int t_in = max(0, min(NB, thin.cols - t0 - NB * c));
  const float* const w_base = wide.X + (w_in > 0 ? w0 + 4 * c : 0);
  const float* const t_base = thin.X + (t_in > 0 ? t0 + NB * c : 0);

  auto entry = [&](const Rows& x, int i) {   // place i's row, -1 for none
    if (i >= s1) return -1;
    const int r = x.index ? x.index[i] : i;
    return r >= 0 && r < x.limit ? r : -1;
  };
  floatx4 acc[4][NB];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

  for (int64_t i0 = (int64_t)s0 + 64 * wave; i0 < s1; i0 += turn) {
    const int rw = entry(wide, (int)(i0 + lane)), rt = entry(thin, (int)(i0 + lane));
    // 16 places a step of four MFMA steps; all of the turn's loads first
    float4 w[4][4];
    float t[4][4][NB];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int r = __shfl(rw, 16 * u + 4 * s + h), q = __shfl(rt, 16 * u + 4 * s + h);
        const bool in = r >= 0 && q >= 0;   // a row that is not there makes its place zero
        const float* x = in ? w_base + (int64_t)r * wide.ld : kZeroChunk;
        const float* y = in ? t_base + (int64_t)q * thin.ld : kZeroChunk;
        if (w_in == 4) {
          w[u][s] = load4(x);
        } else {
          w[u][s] = make_float4(w_in > 0 ? x[0] : 0.f, w_in > 1 ? x[1] : 0.f,
                                w_in > 2 ? x[2] : 0.f, 0.f);
        }
        if (t_in == NB) {
          __builtin_memcpy(t[u][s], y, sizeof(t[u][s]));
        } else {
#pragma unroll
          for (int j = 0; j < NB; ++j) t[u][s][j] = j < t_in ? y[j] : 0.f;
        }
      }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const float4 v = w[u][s];
        const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < NB; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], t[u][s][j], acc[i][j], 0, 0, 0);
      }
  }
  // block (i, j), register r: wide column 4 (4 h + r) + i, thin column NB c + j.  In
  // LDS with C's fast dimension last.
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int a = 4 * (4 * h + r) + i, b = NB * c + j;
        red[wave * kWide * kThin + (kWideA ? a * kThin + b : b * kWide + a)] = acc[i][j][r];
      }
  __syncthreads();
  constexpr int kFast = kWideA ? kThin : kWide;
  const int m0 = kWideA ? w0 : t0, n0 = kWideA ? t0 : w0;
  for (int x = tid; x < kWide * kThin; x += kWaves * 64) {
    const int m = m0 + x / kFast, n = n0 + x % kFast;
    if (m >= p.M || n >= p.N) continue;
    float sum = red[x];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += red[w * kWide * kThin + x];
    if (slices > 1) {
      part[(((int64_t)slice * p.groups + g) * p.M + m) * p.N + n] = sum;
    } else {
      float* out = p.C + g * p.sc + m * p.ldc + n;
      *out = epilogue_apply(ep, sum, out, n);
    }
  }
}

// The slices' sums, added in slice order.
__global__ void __launch_bounds__(256)
    wgrad_join_kernel(GroupedProblem p, Epilogue ep, int slices, const float* __restrict__ part) {
  const int64_t each = (int64_t)p.M * p.N, all = each * p.groups;
  for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < all;
       x += (int64_t)gridDim.x * 256) {
    float sum = 0.f;
    for (int s = 0; s < slices; ++s) sum += part[s * all + x];
    const int64_t g = x / each, y = x - g * each;
    float* out = p.C + g * p.sc + y / p.N * p.ldc + y % p.N;
    *out = epilogue_apply(ep, sum, out, 0);
  }
}

struct ThinPlan {
  bool wide_a;
  int nb, slices;
  int64_t tiles, strips;
};
ThinPlan plan_thin(const GroupedProblem& p) {
  ThinPlan pl;
  pl.wide_a = p.M >= p.N;
  const int64_t wide = pl.wide_a ? p.M : p.N, thin = pl.wide_a ? p.N : p.M;
  pl.nb = thin <= 16 ? 1 : 2;
  pl.tiles = (wide + kWide - 1) / kWide;
  pl.strips = (thin + 16 * pl.nb - 1) / (16 * pl.nb);
  // slices up to one workgroup a CU, of 512 places (a turn of the waves) or more in
  // groups of average size and of 2048 in a group that has nearly all; up to two
  // workgroups a CU where slices of average groups still have 2048 (8192 places of
  // 2048 x 16: 23 us against 35 us for 4 slices; 4096 of 1024 x 64: 18 against 40 for
  // 2; 8 groups of 1024, 2048 x 32: 31 against 36 for 2; 4 of 8192, 2048 x 16: 63 for 4
  // against 74 for 2; 3 groups of 683, 1024 x 8: 11 against 12 for 2)
  const int64_t blocks = pl.tiles * pl.strips * p.groups;
  const int64_t s = std::max(
      std::min(256 / blocks, std::max(p.rows / (512 * (int64_t)p.groups), (int64_t)p.rows / 2048)),
      std::min(512 / blocks, p.rows / (2048 * (int64_t)p.groups)));
  pl.slices = (int)(s < 1 ? 1 : s > kMaxSlices ? kMaxSlices : s);
  return pl;
}

template <int NB, bool kWideA>
void launch(const GroupedProblem& p, const Epilogue& e, const ThinPlan& pl, float* part,
            int64_t blocks, hipStream_t s) {
  hipLaunchKernelGGL((wgrad_thin_kernel<NB, kWideA>), tile_grid(blocks), dim3(kWaves * 64), 0, s, p,
                     e, (int)pl.tiles, (int)pl.strips, pl.slices, part);
}

}  // namespace

hipError_t launch_wgrad_join(const GroupedProblem& p, const Epilogue& e, int slices,
                             const float* part, hipStream_t s) {
  const int64_t all = (int64_t)p.groups * p.M * p.N, wgs = (all + 255) / 256;
  hipLaunchKernelGGL(wgrad_join_kernel, dim3((unsigned)(wgs < 4096 ? wgs : 4096)), dim3(256), 0, s,
                     p, e, slices, part);
  return hipGetLastError();
}

size_t wgrad_thin_floats(const GroupedProblem& p) {
  const ThinPlan pl = plan_thin(p);
  return pl.slices > 1 ? (size_t)pl.slices * p.groups * p.M * p.N : 0;
}

hipError_t launch_wgrad_thin(const GroupedProblem& p, const Epilogue& e, float* part,
                             hipStream_t s) {
  const ThinPlan pl = plan_thin(p);
  const int64_t blocks = pl.tiles * pl.strips * pl.slices * p.groups;
  if (blocks > 0x7fffffff) return hipErrorInvalidConfiguration;
  if (pl.wide_a) {
    pl.nb == 1 ? launch<1, true>(p, e, pl, part, blocks, s)
               : launch<2, true>(p, e, pl, part, blocks, s);
  } else {
    pl.nb == 1 ? launch<1, false>(p, e, pl, part, blocks, s)
               : launch<2, false>(p, e, pl, part, blocks, s);
  }
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || pl.slices == 1) return err;
  return launch_wgrad_join(p, e, pl.slices, part, s);
}

}  // namespace gemmf32
