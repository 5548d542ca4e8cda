// The join of the experts' rows: y_t = sum_j w_tj H[t top + j] + beta y_t, and its
// gradient dH_tj = w_tj dy_t, dw_tj = <dy_t, H_tj>.  Bound by HBM: every row of H is
// read once, every row of Y (of dH) written once: 8192 x 2 rows of 2048 take 41 us (4.8 TB/s,
// a copy's rate) and 55 us (6.2 TB/s), with inputs that the caches do not hold.
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

// `across` threads (a power of two) have four columns each of a token, the workgroups
// behind them the columns beside those.  kAtOnce entries' rows are on the way at once.
__global__ void __launch_bounds__(kThreads)
    join_kernel(JoinProblem p, int across_log2, int blocks) {
  constexpr int kAtOnce = 4;   // (2048 x 8 rows of 2048: 28.7 us, with 2 30.1, with 8 28.0)
  const unsigned id = tile_id(), rows = id / (unsigned)blocks;
  const int64_t t = (int64_t)rows * (kThreads >> across_log2) + (threadIdx.x >> across_log2);
  const int64_t c = 4 * (((int64_t)(id - rows * blocks) << across_log2) +
                         (threadIdx.x & ((1 << across_log2) - 1)));
  if (t >= p.tokens || c >= p.N) return;
  const int n = (int)min((int64_t)4, p.N - c);
  float4 sum{0.f, 0.f, 0.f, 0.f};
  for (int first = 0; first < p.top; first += kAtOnce) {
    const int64_t i = t * p.top + first;
    const int here = min(kAtOnce, p.top - first);
    bool there[kAtOnce];
    float w[kAtOnce];
    float4 h[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      there[j] = j < here && counts(p, i + j);
      w[j] = j < here ? p.weight[i + j] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      if (there[j]) h[j] = load_part(p.H + (i + j) * p.ldh + c, n);
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      if (there[j]) add(sum, w[j], h[j]);
  }
  float* y = p.Y + t * p.ldy + c;
  if (p.beta != 0.f) add(sum, p.beta, load_part(y, n));
  store_part(y, sum, n);
}

// One wave an entry; kAtOnce of its steps along the columns on the way at once.
__global__ void __launch_bounds__(kThreads) join_grad_kernel(JoinProblem p) {
  constexpr int kAtOnce = 4, kStep = 4 * 64;
  const int lane = threadIdx.x & 63;
  const int64_t i = (int64_t)tile_id() * (kThreads / 64) + (threadIdx.x >> 6);
  if (i >= p.tokens * p.top) return;
  const bool there = counts(p, i);
  const float w = there ? p.weight[i] : 0.f;
  const float *dy = p.dY + (uint32_t)i / (uint32_t)p.top * p.lddy, *h = p.H + i * p.ldh;
  float* dh = p.dH + i * p.lddh;
  float dot = 0.f;
  auto one = [&](float* to, float4 g, float4 x, int n) {
    float4 d{0.f, 0.f, 0.f, 0.f};
    dot += g.x * x.x + g.y * x.y + (g.z * x.z + g.w * x.w);
    add(d, w, g);
    store_part(to, d, n);
  };
  int64_t c = 4 * lane;
  if (!there) {
    for (; c < p.N; c += kStep)
      store_part(dh + c, float4{0.f, 0.f, 0.f, 0.f}, (int)min((int64_t)4, p.N - c));
  }
  for (; c + (kAtOnce - 1) * kStep + 4 <= p.N; c += kAtOnce * kStep) {
    float4 g[kAtOnce], x[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      g[k] = load_part(dy + c + k * kStep, 4);
      x[k] = load_part(h + c + k * kStep, 4);
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) one(dh + c + k * kStep, g[k], x[k], 4);
  }
  for (; c < p.N; c += kStep) {
    const int n = (int)min((int64_t)4, p.N - c);
    one(dh + c, load_part(dy + c, n), load_part(h + c, n), n);
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
  const int blocks = (p.N + (4 << log2) - 1) / (4 << log2);
  const dim3 grid = tile_grid((p.tokens + per - 1) / per * blocks);
  join_kernel<<<grid, kThreads, 0, s>>>(p, log2, blocks);
  return hipGetLastError();
}

hipError_t launch_join_grad(const JoinProblem& p, hipStream_t s) {
  const int64_t per = kThreads / 64, entries = p.tokens * p.top;
  join_grad_kernel<<<tile_grid((entries + per - 1) / per), kThreads, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace gemmf32
