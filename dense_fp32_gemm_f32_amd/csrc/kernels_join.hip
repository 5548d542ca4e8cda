// The join of the experts' rows: y_t = sum_j w_tj H[t top + j] + beta y_t, and its
// gradient dH_tj = w_tj dy_t, dw_tj = <dy_t, H_tj>.  Bound by HBM: every row of H is
// read once, every row of Y (of dH) written once.
#include "experts_internal.h"

namespace gemmf32 {
namespace {

constexpr int kThreads = 256;

// Up to four floats from or to a 4-byte aligned address: `n` of them are there.
__device__ __forceinline__ float4 load_part(const float* p, int n) {
  float4 v{0.f, 0.f, 0.f, 0.f};
  if (n >= 4) {
    __builtin_memcpy(&v, p, sizeof(v));
  } else {
    v.x = p[0];
    if (n > 1) v.y = p[1];
    if (n > 2) v.z = p[2];
  }
  return v;
}
__device__ __forceinline__ void store_part(float* p, float4 v, int n) {
  if (n >= 4) {
    __builtin_memcpy(p, &v, sizeof(v));
  } else {
    p[0] = v.x;
    if (n > 1) p[1] = v.y;
    if (n > 2) p[2] = v.z;
  }
}
__device__ __forceinline__ void add(float4& a, float w, float4 b) {
  a.x += w * b.x;
  a.y += w * b.y;
  a.z += w * b.z;
  a.w += w * b.w;
}

__device__ __forceinline__ bool counts(const JoinProblem& p, int64_t i) {
  if (!p.choice) return true;
  const int c = p.choice[i];
  return c >= 0 && c < p.groups;
}

// `across` threads (a power of two) go along a token's columns, four each.
__global__ void __launch_bounds__(kThreads) join_kernel(JoinProblem p, int across_log2) {
  const int across = 1 << across_log2;
  const int64_t t = (int64_t)tile_id() * (kThreads >> across_log2) + (threadIdx.x >> across_log2);
  if (t >= p.tokens) return;
  for (int64_t c = 4 * (int64_t)(threadIdx.x & (across - 1)); c < p.N; c += 4 * across) {
    const int n = (int)min((int64_t)4, p.N - c);
    float4 sum{0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < p.top; ++j) {
      const int64_t i = t * p.top + j;
      if (counts(p, i)) add(sum, p.weight[i], load_part(p.H + i * p.ldh + c, n));
    }
    float* y = p.Y + t * p.ldy + c;
    if (p.beta != 0.f) add(sum, p.beta, load_part(y, n));
    store_part(y, sum, n);
  }
}

// One wave an entry.
__global__ void __launch_bounds__(kThreads) join_grad_kernel(JoinProblem p) {
  const int lane = threadIdx.x & 63;
  const int64_t i = (int64_t)tile_id() * (kThreads / 64) + (threadIdx.x >> 6);
  if (i >= p.tokens * p.top) return;
  const bool there = counts(p, i);
  const float w = there ? p.weight[i] : 0.f;
  const float* dy = p.dY + i / p.top * p.lddy;
  float dot = 0.f;
  for (int64_t c = 4 * lane; c < p.N; c += 4 * 64) {
    const int n = (int)min((int64_t)4, p.N - c);
    float4 d{0.f, 0.f, 0.f, 0.f};
    if (there) {
      const float4 g = load_part(dy + c, n), h = load_part(p.H + i * p.ldh + c, n);
      dot += g.x * h.x + g.y * h.y + (g.z * h.z + g.w * h.w);
      add(d, w, g);
    }
    store_part(p.dH + i * p.lddh + c, d, n);
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) dot += __shfl_xor(dot, d);
  if (lane == 0) p.dweight[i] = dot;
}

}  // namespace

hipError_t launch_join(const JoinProblem& p, hipStream_t s) {
  int log2 = 3;   // at least 8 threads, 128 bytes, along the columns
  while ((4 << log2) < p.N && (1 << log2) < kThreads) ++log2;
  const int64_t per = kThreads >> log2;
  join_kernel<<<tile_grid((p.tokens + per - 1) / per), kThreads, 0, s>>>(p, log2);
  return hipGetLastError();
}

hipError_t launch_join_grad(const JoinProblem& p, hipStream_t s) {
  const int64_t per = kThreads / 64, entries = p.tokens * p.top;
  join_grad_kernel<<<tile_grid((entries + per - 1) / per), kThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace gemmf32
