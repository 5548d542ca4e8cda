// Routing to experts and its gradient, one wave a token, logits in registers
// (expert i 64 + lane in register i).
//
// Which experts are chosen is decided in 64 bits: scores that 32 bits would round
// onto each other, or exchange, go by their real order.  The weights and the
// gradient are fp32; renormalised softmax weights are the softmax of the chosen
// logits alone, so they hold where the chosen scores would underflow.
#include "experts_internal.h"

#include <cfloat>

namespace gemmf32 {
namespace {

constexpr int kWaves = 4, kThreads = kWaves * 64;

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor(x, d));
  return x;
}
template <class T>
__device__ __forceinline__ T wave_sum(T x) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
  return x;
}

// The largest of the wave's 64 E values and its number i 64 + lane, the lowest of
// equal ones; -1 where all are -infinity.
template <int E>
__device__ __forceinline__ int wave_best(const double (&v)[E], int lane, double& best) {
  double x = v[0];
  int at = lane;
#pragma unroll
  for (int i = 1; i < E; ++i)
    if (v[i] > x) {
      x = v[i];
      at = i * 64 + lane;
    }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const double y = __shfl_xor(x, d);
    const int yat = __shfl_xor(at, d);
    if (y > x || (y == x && yat < at)) {
      x = y;
      at = yat;
    }
  }
  best = x;
  return x > -INFINITY ? at : -1;
}

// Lanes of one wave pass values through LDS.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A token's logits: NaN and -infinity (and what is past the end) as -infinity,
// +infinity as the largest finite value.
template <int E>
__device__ __forceinline__ void load_logits(const RouteProblem& p, int64_t t, int lane,
                                            float (&l)[E]) {
  const float* row = p.logits + t * p.ldl;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int e = i * 64 + lane;
    const float x = e < p.experts ? row[e] : -INFINITY;
    l[i] = x > -INFINITY ? fminf(x, FLT_MAX) : -INFINITY;
  }
}

// Softmax of the wave's logits into s; all -infinity gives zeros.
template <int E>
__device__ __forceinline__ void softmax(const float (&l)[E], float (&s)[E]) {
  float m = l[0];
#pragma unroll
  for (int i = 1; i < E; ++i) m = fmaxf(m, l[i]);
  m = wave_max(m);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    s[i] = l[i] > -INFINITY ? expf(l[i] - m) : 0.f;
    sum += s[i];
  }
  sum = wave_sum(sum);
#pragma unroll
  for (int i = 0; i < E; ++i) s[i] = sum > 0.f ? s[i] / sum : 0.f;
}

// The choices in 64 bits: lane j gets the expert of choice j (-1: none).
template <int E>
__device__ __forceinline__ int choose(const RouteProblem& p, const float (&l)[E], int lane,
                                      double* lds) {
  double s[E], v[E];
  const bool grouped = p.group_top < p.groups;
  if (p.bias || (grouped && p.group_best == 2)) {
    if (p.sigmoid) {
#pragma unroll
      for (int i = 0; i < E; ++i) s[i] = 1.0 / (1.0 + exp(-(double)l[i]));
    } else {
      float m = l[0];
#pragma unroll
      for (int i = 1; i < E; ++i) m = fmaxf(m, l[i]);
      m = wave_max(m);
      double sum = 0;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        s[i] = l[i] > -INFINITY ? exp((double)l[i] - (double)m) : 0.0;
        sum += s[i];
      }
      sum = wave_sum(sum);
#pragma unroll
      for (int i = 0; i < E; ++i) s[i] = sum > 0 ? s[i] / sum : 0.0;
    }
  }
#pragma unroll
  for (int i = 0; i < E; ++i) {
    v[i] = l[i];   // without a bias the scores have the logits' order
    if (p.bias && l[i] > -INFINITY) {
      const float b = p.bias[i * 64 + lane];
      const double x = s[i] + (double)(b > FLT_MAX ? FLT_MAX : b);   // NaN stays NaN
      v[i] = x > -INFINITY ? x : -INFINITY;
    }
  }
  if (grouped) {
    // a group's score by one lane each, then the best groups, marked in LDS
    const int size = p.experts / p.groups;
    const bool sums = p.group_best == 2;
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i * 64 + lane < p.experts)
        lds[i * 64 + lane] = sums && !p.bias ? (v[i] > -INFINITY ? s[i] : -INFINITY) : v[i];
    wave_fence();
    double gs[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int g = i * 64 + lane;
      double a = -INFINITY, b = -INFINITY;
      if (g < p.groups)
        for (int k = 0; k < size; ++k) {
          const double x = lds[g * size + k];
          if (x > a) {
            b = a;
            a = x;
          } else if (x > b) {
            b = x;
          }
        }
      gs[i] = sums && b > -INFINITY ? a + b : a;
    }
    wave_fence();
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i * 64 + lane < p.groups) lds[i * 64 + lane] = 0;
    for (int j = 0; j < p.group_top; ++j) {
      double best;
      const int g = wave_best<E>(gs, lane, best);
      if (g < 0) break;
      if (lane == 0) lds[g] = 1;
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (i * 64 + lane == g) gs[i] = -INFINITY;
    }
    wave_fence();
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i * 64 + lane < p.experts && lds[(i * 64 + lane) / size] == 0) v[i] = -INFINITY;
  }
  int mine = -1;
  for (int j = 0; j < p.top; ++j) {
    double best;
    const int e = wave_best<E>(v, lane, best);
    if (e < 0) break;
    if (lane == j) mine = e;
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i * 64 + lane == e) v[i] = -INFINITY;
  }
  return mine;
}

// Softmax over the lanes' logits x of those with a choice (0 for the others).
__device__ __forceinline__ float share_of_chosen(float x, bool there) {
  const float m = wave_max(there ? x : -INFINITY);
  const float q = there ? expf(x - m) : 0.f;
  const float sum = wave_sum(q);
  return there ? q / sum : 0.f;
}

// Renormalised sigmoid scores, for sums that underflow as a softmax: far below
// zero the sigmoid is the exponential.
__device__ __forceinline__ float share_of_sigmoid(float x, float s, bool there) {
  const float sum = wave_sum(there ? s : 0.f);
  if (sum < 1e-30f) return share_of_chosen(x, there);
  return there ? s / sum : 0.f;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

template <int E>
__global__ void __launch_bounds__(kThreads) route_kernel(RouteProblem p) {
  __shared__ double lds[kWaves][64 * E];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t t = (int64_t)tile_id() * kWaves + wave;
  if (t >= p.tokens) return;
  float l[E];
  load_logits<E>(p, t, lane, l);
  const int e = choose<E>(p, l, lane, lds[wave]);
  const bool there = e >= 0;
  float x = 0.f, w;   // this lane's chosen logit
  if (there) x = fminf(p.logits[t * p.ldl + e], FLT_MAX);
  if (p.sigmoid) {
    w = there ? sigmoid(x) : 0.f;
    if (p.renorm) w = share_of_sigmoid(x, w, there);
  } else if (p.renorm) {
    w = share_of_chosen(x, there);
  } else {
    float s[E];
    softmax<E>(l, s);
    w = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float y = __shfl(s[i], e & 63);
      if (there && e >> 6 == i) w = y;
    }
  }
  if (lane < p.top) {
    p.choice[t * p.top + lane] = e;
    p.weight[t * p.top + lane] = there ? p.scale * w : 0.f;
  }
}

// With g = scale dw at the chosen experts (0 elsewhere) and sums over the chosen:
//   softmax        dl_i = p_i (g_i - sum p_k g_k)
//   renormalised   dl_i = q_i (g_i - sum q_k g_k), q the shares of the chosen
//   sigmoid        dl_i = s_i (1 - s_i) g_i
//   renormalised   dl_i = q_i (1 - s_i) (g_i - sum q_k g_k)
// Lane j forms the gradient of choice j; it is handed to the expert's lane choice
// by choice, so an expert named twice gets both.
template <int E>
__global__ void __launch_bounds__(kThreads) route_grad_kernel(RouteProblem p) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t t = (int64_t)tile_id() * kWaves + wave;
  if (t >= p.tokens) return;
  const float* row = p.logits + t * p.ldl;
  int e = lane < p.top ? p.choice[t * p.top + lane] : -1;
  float x = e >= 0 && e < p.experts ? row[e] : -INFINITY;
  const bool there = x > -INFINITY;
  x = fminf(x, FLT_MAX);
  const float g = there ? p.scale * p.dweight[t * p.top + lane] : 0.f;
  float d[E];
#pragma unroll
  for (int i = 0; i < E; ++i) d[i] = 0.f;
  float mine;
  if (!p.sigmoid && !p.renorm) {
    float l[E], s[E];
    load_logits<E>(p, t, lane, l);
    softmax<E>(l, s);
    mine = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float y = __shfl(s[i], e & 63);
      if (there && e >> 6 == i) mine = y;
    }
    mine *= g;
    const float dot = wave_sum(mine);
#pragma unroll
    for (int i = 0; i < E; ++i) d[i] = l[i] > -INFINITY ? -s[i] * dot : 0.f;
  } else {
    const float s = p.sigmoid && there ? sigmoid(x) : 0.f;
    if (p.renorm) {
      const float q = p.sigmoid ? share_of_sigmoid(x, s, there) : share_of_chosen(x, there);
      mine = q * (g - wave_sum(there ? q * g : 0.f)) * (1.f - s);
    } else {
      mine = s * (1.f - s) * g;
    }
  }
  for (int j = 0; j < p.top; ++j) {
    const int to = __builtin_amdgcn_readlane(there ? e : -1, j);
    const float y = __shfl(mine, j);
    if (to < 0) continue;
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i * 64 + lane == to) d[i] += y;
  }
  float* out = p.dlogits + t * p.lddl;
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (i * 64 + lane < p.experts) out[i * 64 + lane] = d[i];
}

template <template <int> class K>
hipError_t by_size(const RouteProblem& p, hipStream_t s) {
  if (p.experts <= 64) return K<1>::run(p, s);
  if (p.experts <= 128) return K<2>::run(p, s);
  if (p.experts <= 256) return K<4>::run(p, s);
  if (p.experts <= 512) return K<8>::run(p, s);
  return K<16>::run(p, s);
}
template <int E>
struct Route {
  static hipError_t run(const RouteProblem& p, hipStream_t s) {
    route_kernel<E><<<tile_grid(((int64_t)p.tokens + kWaves - 1) / kWaves), kThreads, 0, s>>>(p);
    return hipGetLastError();
  }
};
template <int E>
struct RouteGrad {
  static hipError_t run(const RouteProblem& p, hipStream_t s) {
    route_grad_kernel<E>
        <<<tile_grid(((int64_t)p.tokens + kWaves - 1) / kWaves), kThreads, 0, s>>>(p);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_route(const RouteProblem& p, hipStream_t s) { return by_size<Route>(p, s); }
hipError_t launch_route_grad(const RouteProblem& p, hipStream_t s) {
  return by_size<RouteGrad>(p, s);
}

}  // namespace gemmf32
