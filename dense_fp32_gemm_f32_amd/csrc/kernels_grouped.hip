// Products whose rows belong to different weights (gfx950): for every place i
// of group g, C[ic(i)] = act(alpha s_g A[ia(i)] op(B_g) + beta C[ic(i)] + bias_g),
// and the gradient of the weights, C_g = alpha sum_i A[ia(i)]^T B[ib(i)] + beta C_g.
//
// The group sizes are known on the device only, so the grid covers the most row
// tiles that the places can need and each workgroup finds its tile from the
// offsets.  64 x 64 tiles, 4 waves of one 32 x 32 MFMA block, K-tiles of 16
// staged through registers into LDS with every element guarded: any size,
// pitch and alignment.
#include "grouped_internal.h"
#include "mfma_common.h"

namespace gemmf32 {
namespace {

using namespace mfma;

constexpr int kT = 64, kBK = 16, kPad = 4;

// One K-tile of an operand: 64 rows (of A, or columns of op(B)) by 16 k in LDS
// as [k][row], fetched by get(row, k).
template <class Get>
__device__ __forceinline__ void stage(float (*lds)[kT + kPad], bool row_fast, Get get) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int v = 0; v < kT * kBK / 256; ++v) {
    const int e = v * 256 + tid;
    const int r = row_fast ? e % kT : e / kBK;
    const int k = row_fast ? e / kT : e % kBK;
    lds[k][r] = get(r, k);
  }
}

__device__ __forceinline__ void multiply(floatx16& acc, const float (*la)[kT + kPad],
                                         const float (*lb)[kT + kPad], int wave, int lane) {
  const int wm = (wave & 1) * 32, wn = (wave >> 1) * 32, lr = lane & 31, lk = lane >> 5;
#pragma unroll
  for (int k = 0; k < kBK; k += 2)
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(la[k + lk][wm + lr], lb[k + lk][wn + lr], acc, 0,
                                               0, 0);
}

__global__ void __launch_bounds__(256)
    grouped_kernel(GroupedProblem p, Epilogue ep, int tiles_n, unsigned cap) {
  __shared__ float la[kBK][kT + kPad], lb[kBK][kT + kPad];
  __shared__ int row_a[kT], row_c[kT];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  RowTiles rt{p.offsets, p.groups, p.rows, kT, lane, cap, 0};
  const unsigned total = rt.total();
  const unsigned id = tile_id();
  const unsigned t = id / tiles_n;
  int g = 0, begin = 0, end = 0;
  unsigned first = 0;
  if (t >= total || !rt.find(t, g, begin, end, first)) return;
  const int m0 = begin + (int)(t - first) * kT, n0 = (int)(id % tiles_n) * kT;
  if (tid < kT) {
    const int i = m0 + tid;
    int a = -1, c = -1;
    if (i < end) {
      a = p.ia ? p.ia[i] : i;
      c = p.ic ? p.ic[i] : i;
      if (a < 0 || a >= p.rows_a) a = -1;
      if (c < 0 || c >= p.rows_c) c = -1;
    }
    row_a[tid] = a;
    row_c[tid] = c;
  }
  const float* B = p.B + g * p.sb;
  floatx16 acc = {};
  for (int k0 = 0; k0 < p.K; k0 += kBK) {
    __syncthreads();
    stage(la, false, [&](int r, int k) {
      const int a = row_a[r];
      return a >= 0 && k0 + k < p.K ? p.A[a * p.lda + k0 + k] : 0.f;
    });
    stage(lb, !p.tb, [&](int r, int k) {
      if (n0 + r >= p.N || k0 + k >= p.K) return 0.f;
      return p.tb ? B[(n0 + r) * p.ldb + k0 + k] : B[(k0 + k) * p.ldb + n0 + r];
    });
    __syncthreads();
    multiply(acc, la, lb, wave, lane);
  }
  __syncthreads();
  const float scale = p.gscale ? p.gscale[g] : 1.f;
  if (ep.bias) ep.bias += g * p.sbias;
  const int col = n0 + (wave >> 1) * 32 + (lane & 31);
  if (col >= p.N) return;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int c = row_c[(wave & 1) * 32 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)];
    if (c < 0) continue;
    float* out = p.C + c * p.ldc + col;
    *out = epilogue_apply(ep, scale * acc[r], out, col);
  }
}

__global__ void __launch_bounds__(256)
    grouped_wgrad_kernel(GroupedProblem p, Epilogue ep, int tiles_n) {
  __shared__ float la[kBK][kT + kPad], lb[kBK][kT + kPad];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int g = blockIdx.y;
  int begin, end;
  group_span(p.offsets, g, p.rows, begin, end);
  const int m0 = (int)(blockIdx.x / tiles_n) * kT, n0 = (int)(blockIdx.x % tiles_n) * kT;
  floatx16 acc[1][1] = {};
  for (int i0 = begin; i0 < end; i0 += kBK) {
    __syncthreads();
    stage(la, true, [&](int r, int k) {
      if (m0 + r >= p.M || k >= end - i0) return 0.f;
      const int a = p.ia ? p.ia[i0 + k] : i0 + k;
      return a >= 0 && a < p.rows_a ? p.A[a * p.lda + m0 + r] : 0.f;
    });
    stage(lb, true, [&](int r, int k) {
      if (n0 + r >= p.N || k >= end - i0) return 0.f;
      const int b = p.ib ? p.ib[i0 + k] : i0 + k;
      return b >= 0 && b < p.rows_b ? p.B[b * p.ldb + n0 + r] : 0.f;
    });
    __syncthreads();
    multiply(acc[0][0], la, lb, wave, lane);
  }
  store_blocks<1, 1>(acc, p.C + g * p.sc, p.ldc, p.M, p.N,
                     m0 + (wave & 1) * 32, n0 + (wave >> 1) * 32, lane, false, ep);
}

}  // namespace

hipError_t launch_grouped(const GroupedProblem& p, const Epilogue& e, hipStream_t s) {
  const int64_t tiles_n = (p.N + kT - 1) / kT;
  const int64_t cap = most_row_tiles(p.rows, p.groups, kT);
  if (cap * tiles_n > 0x7fffffff) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(grouped_kernel, tile_grid(cap * tiles_n), dim3(256), 0, s, p, e,
                     (int)tiles_n, (unsigned)cap);
  return hipGetLastError();
}

hipError_t launch_grouped_wgrad(const GroupedProblem& p, const Epilogue& e, hipStream_t s) {
  const int64_t tiles_n = (p.N + kT - 1) / kT, tiles_m = (p.M + kT - 1) / kT;
  if (tiles_m * tiles_n > kGridX) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(grouped_wgrad_kernel, dim3((unsigned)(tiles_m * tiles_n), (unsigned)p.groups),
                     dim3(256), 0, s, p, e, (int)tiles_n);
  return hipGetLastError();
}

}  // namespace gemmf32
