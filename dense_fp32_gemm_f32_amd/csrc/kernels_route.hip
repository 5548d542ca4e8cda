// Routing to experts and its gradient, one wave a token, the logits in registers:
// lane l has experts l E to l E + E - 1, so that the lowest lane is the lowest expert.
//
// Which experts are chosen is decided as if in 64 bits: scores that 32 bits would round
// onto each other, or exchange, go by their real order.  Without a bias the logits
// themselves have that order.  With one (or sums of scores for groups) the scores are
// formed in 32 bits first; where two that decide something lie within the error of
// that, the token is done again in 64 bits.  The weights and the gradient are fp32;
// renormalised softmax weights are the softmax of the chosen logits alone, so they
// hold where the chosen scores would underflow.
//
// Each lane sorts its keys once; a choice is then the largest head of 64 lists, six DPP
// steps and a pop.  Bound by the vector instructions: 16384 x 256, 8 choices, take 12 us
// without a bias, 15 with one, 18 with the best 4 of 8 groups (54 where every choice was
// made in 64 bits); the read of the logits alone would take 3.5.  Groups that are no whole
// number of lanes are done in 64 bits from the start: 16384 x 144 in 8 groups take 73 us.
#include "experts_internal.h"

#include <cfloat>
#include <climits>

namespace gemmf32 {
namespace {

constexpr int kWaves = 4, kThreads = kWaves * 64;

typedef float f32x4 __attribute__((ext_vector_type(4)));

// x of the lane that kCtrl names; none's in rows of 16 outside kRows.
template <int kCtrl, int kRows, class T>
__device__ __forceinline__ T dpp(T none, T x) {
  return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none),
                                                           __builtin_bit_cast(int, x), kCtrl,
                                                           kRows, 0xf, false));
}

// op over the wave's values, none being its neutral one: lanes 1, 2, then (as fours,
// and then eights, agree by now) the mirrored half row and row, then row 0 (2) into
// row 1 (3), and both into row 3, whose last lane has it.
template <class T, class Op>
__device__ __forceinline__ T wave_all(T x, T none, Op op) {
  x = op(x, dpp<0xb1, 0xf>(none, x));
  x = op(x, dpp<0x4e, 0xf>(none, x));
  x = op(x, dpp<0x141, 0xf>(none, x));
  x = op(x, dpp<0x140, 0xf>(none, x));
  x = op(x, dpp<0x142, 0xa>(none, x));
  x = op(x, dpp<0x143, 0xc>(none, x));
  return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}
__device__ __forceinline__ int wave_max(int x) {
  return wave_all(x, INT_MIN, [](int a, int b) { return a > b ? a : b; });
}
__device__ __forceinline__ float wave_sum(float x) {
  return wave_all(x, 0.f, [](float a, float b) { return a + b; });
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
  return x;
}

// Floats that are not NaN as integers of the same order, 0 and -0 alike; kNone for what
// is not to be chosen, -infinity too.
constexpr int kNone = INT_MIN;
__device__ __forceinline__ int key_of(float x) {
  const int i = __float_as_int(x + 0.f);
  return x > -INFINITY ? i ^ (i >> 31 & 0x7fffffff) : kNone;
}
__device__ __forceinline__ float of_key(int k) {
  return k == kNone ? -INFINITY : __int_as_float(k ^ (k >> 31 & 0x7fffffff));
}
__device__ __forceinline__ float wave_max(float x) { return of_key(wave_max(key_of(x))); }

// mask (0 or -1) ? a : b, in one instruction; of array elements a conditional would
// become a choice of their index.
__device__ __forceinline__ int pick(int mask, int a, int b) { return (a & mask) | (b & ~mask); }

__device__ __forceinline__ float lane_value(float x, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}

// The largest of the wave's 64 E values and its number, the lowest of equal ones; -1
// where all are -infinity.
template <int E>
__device__ __forceinline__ int wave_best(const double (&v)[E], int lane) {
  double x = v[0];
  int at = lane * E;
#pragma unroll
  for (int i = 1; i < E; ++i)
    if (v[i] > x) {
      x = v[i];
      at = lane * E + i;
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
  return x > -INFINITY ? at : -1;
}

// Lanes of one wave pass values through LDS.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A lane's share of a row of n values, E from lane E on; past the end what is given.
// (Loads without a branch: past the end they read the last values.)
template <int E>
__device__ __forceinline__ void load_row(const float* row, int n, int lane, float past,
                                         float (&v)[E]) {
  const int first = lane * E;
  if (E >= 4 && n % 4 == 0 && n > 0 && reinterpret_cast<uintptr_t>(row) % 16 == 0) {
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(row + min(first + i, n - 4));
#pragma unroll
      for (int k = 0; k < 4 && i + k < E; ++k) v[i + k] = first + i < n ? x[k] : past;
    }
  } else if (n > 0) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float x = row[min(first + i, n - 1)];
      v[i] = first + i < n ? x : past;
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = past;
  }
}

template <int E>
__device__ __forceinline__ void store_row(float* row, int n, int lane, const float (&v)[E]) {
  const int first = lane * E;
  if constexpr (E >= 4) {
    if (n % 4 == 0 && reinterpret_cast<uintptr_t>(row) % 16 == 0) {
#pragma unroll
      for (int i = 0; i < E; i += 4)
        if (first + i < n)
          *reinterpret_cast<f32x4*>(row + first + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (first + i < n) row[first + i] = v[i];
}

// A token's logits: NaN and -infinity (and what is past the end) as -infinity,
// +infinity as the largest finite value.
template <int E>
__device__ __forceinline__ void load_logits(const RouteProblem& p, int64_t t, int lane,
                                            float (&l)[E]) {
  load_row<E>(p.logits + t * p.ldl, p.experts, lane, -INFINITY, l);
#pragma unroll
  for (int i = 0; i < E; ++i) l[i] = l[i] > -INFINITY ? fminf(l[i], FLT_MAX) : -INFINITY;
}

template <int E>
__device__ __forceinline__ float largest(const float (&l)[E]) {
  float m = l[0];
#pragma unroll
  for (int i = 1; i < E; ++i) m = fmaxf(m, l[i]);
  return wave_max(m);
}

// The sum of exp(l - m), m the largest; all -infinity gives 0.
template <int E>
__device__ __forceinline__ float exp_sum(const float (&l)[E], float m) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) sum += l[i] > -INFINITY ? expf(l[i] - m) : 0.f;
  return wave_sum(sum);
}

// Keys and their numbers from the largest down, the lower number first of equal ones
// (an odd-even merge sort).
template <int E>
__device__ __forceinline__ void sort_down(int (&v)[E], int (&at)[E]) {
#pragma unroll
  for (int p = 1; p < E; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < E; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i) {
          const int x = i + j, y = i + j + k;
          if (y < E && x / (2 * p) == y / (2 * p)) {
            const int vx = v[x], vy = v[y], ax = at[x], ay = at[y];
            const int swap = -(int)((vy > vx) | ((vy == vx) & (ay < ax)));
            v[x] = max(vx, vy);
            v[y] = min(vx, vy);
            at[x] = pick(swap, ay, ax);
            at[y] = pick(swap, ax, ay);
          }
        }
}

// What 32-bit scores s + bias have to differ by for their order to be the real one.
// A sigmoid is off by less than 2^-22: 0.45 2^-23 by the exponential (one unit of its
// last place, and 2^-23 of its argument x, where x s (1 - s) < 0.23), half a unit by the
// sum, one by the reciprocal.  A softmax's scores share the sum's error: 21 roundings of
// half a unit, and the exponentials' mean one (below 7 units: the mean of |x| is below
// 4.5 for 1024 experts); with 3 units of their own, two differ rightly to within 2^-18
// of the largest score.  The addition of the bias rounds once.
struct Margin {
  float score;   // of the difference of two scores
  __device__ __forceinline__ bool apart(float above, float below) const {
    return above - below > score + 0x1p-22f * fmaxf(fabsf(above), fabsf(below));
  }
  // What a group's score a + b is off by: the additions of the bias by 2^-24 of |a| and of
  // |b|, which the sum may be far below, their own by 2^-24 of that; as much again covers
  // the rounding of what it is added to.  Of two groups' four scores' errors, half.
  __device__ __forceinline__ float of_group(float a, float b) const {
    return score + 0x1p-22f * (fabsf(a) + fabsf(b));
  }
};

// A token's scores in 64 bits.
template <int E>
struct Exact {
  const RouteProblem& p;
  double m = 0, sum = 1;   // of a softmax
  __device__ __forceinline__ Exact(const RouteProblem& p, const float (&l)[E]) : p(p) {
    if (p.sigmoid) return;
    m = largest<E>(l);
    sum = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) sum += l[i] > -INFINITY ? exp(l[i] - m) : 0.0;
    sum = wave_sum(sum);
  }
  __device__ __forceinline__ double score(double l) const {
    return p.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - m) / sum;
  }
  // With the bias, of a logit above -infinity; one that is not to be chosen -infinity.
  __device__ __forceinline__ double biased(double l, float b) const {
    const double x = score(l) + (double)(b > FLT_MAX ? FLT_MAX : b);   // NaN stays NaN
    return x > -INFINITY ? x : -INFINITY;
  }
};

// Whether the group that lane g has the score of is above this lane's, by lane g.
__device__ __forceinline__ bool above(double other, double mine, int g, int lane) {
  return (other > mine) | ((other == mine) & (g < lane));
}
__device__ __forceinline__ double lane_value(double x, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)u, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Whether lane g's group is among the best, by scores in 64 bits: as choose_fast finds it.
template <int E>
__device__ __forceinline__ bool in_best_groups(const RouteProblem& p, const float (&l)[E],
                                               int lanes, int lane, double* lds) {
  const Exact<E> exact(p, l);
  float bias[E];
  if (p.bias) load_row<E>(p.bias, p.experts, lane, 0.f, bias);
  double a = -INFINITY, b = -INFINITY;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    double x = -INFINITY;
    if (l[i] > -INFINITY) x = p.bias ? exact.biased(l[i], bias[i]) : exact.score(l[i]);
    b = fmax(b, fmin(a, x));
    a = fmax(a, x);
  }
  wave_fence();
  lds[2 * lane] = a;
  lds[2 * lane + 1] = b;
  wave_fence();
  a = b = -INFINITY;
  if (lane < p.groups)
    for (int k = 0; k < lanes; ++k) {
      const double x = lds[2 * (lane * lanes + k)], y = lds[2 * (lane * lanes + k) + 1];
      b = fmax(fmax(b, y), fmin(a, x));
      a = fmax(a, x);
    }
  const double score = p.group_best == 2 && b > -INFINITY ? a + b : a;
  int rank = 0;
  for (int g = 0; g < p.groups; ++g) rank += above(lane_value(score, g), score, g, lane);
  return rank < p.group_top;
}

// The choices by 32-bit scores: lane j gets the expert of choice j (-1: none).  False
// where these do not decide them.
template <int E>
__device__ __forceinline__ bool choose_fast(const RouteProblem& p, const float* row,
                                            const float (&l)[E], int lane, double* lds,
                                            int& mine) {
  const bool grouped = p.group_top < p.groups, sums = p.group_best == 2;
  const bool scores = p.bias || (grouped && sums);
  float s[E];
  int v[E];
  Margin margin = {0x1.8p-21f};
  if (scores) {
    constexpr float kLog2e = 1.44269504f;
    if (p.sigmoid) {
#pragma unroll
      for (int i = 0; i < E; ++i)
        s[i] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(l[i] * -kLog2e));
    } else {
      const float m = largest<E>(l);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        s[i] = l[i] > -INFINITY ? __builtin_amdgcn_exp2f((l[i] - m) * kLog2e) : 0.f;
        sum += s[i];
      }
      const float r = __builtin_amdgcn_rcpf(wave_sum(sum));
      margin.score = 0x1p-18f * r;
#pragma unroll
      for (int i = 0; i < E; ++i) s[i] *= r;
    }
  }
  if (p.bias) {
    float b[E];
    load_row<E>(p.bias, p.experts, lane, 0.f, b);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float x = s[i] + fminf(b[i], FLT_MAX);
      v[i] = ((l[i] > -INFINITY) & (b[i] > -INFINITY)) ? key_of(x) : kNone;   // NaN: neither
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = key_of(l[i]);
  }
  if (grouped) {
    // whole lanes to a group: each lane's best two, then those of a group by one lane
    const int size = p.group_size, lanes = size / E;
    if (lanes * E != size) return false;
    int a = kNone, b = kNone;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      int x = v[i];
      if (sums && !p.bias) x = x != kNone ? key_of(s[i]) : kNone;
      b = max(b, min(a, x));
      a = max(a, x);
    }
    int* const best = reinterpret_cast<int*>(lds);
    best[2 * lane] = a;
    best[2 * lane + 1] = b;
    wave_fence();
    a = b = kNone;
    if (lane < p.groups)
      for (int k = 0; k < lanes; ++k) {
        const int x = best[2 * (lane * lanes + k)], y = best[2 * (lane * lanes + k) + 1];
        b = max(max(b, y), min(a, x));
        a = max(a, x);
      }
    // (a sum that passes the largest float stays above kNone: a group of the lowest biases
    // comes before one without an expert; which of such sums is above, 64 bits decide)
    const bool both = sums && b != kNone;
    const float sum = fminf(fmaxf(of_key(a) + of_key(b), -FLT_MAX), FLT_MAX);
    const int score = both ? key_of(sum) : a;
    int rank = 0;   // groups above this lane's
    for (int g = 0; g < p.groups; ++g) {
      const int other = __builtin_amdgcn_readlane(score, g);
      rank += (other > score) | ((other == score) & (g < lane));
    }
    bool in = rank < p.group_top;
    if (scores) {
      // each group's score lies within `off` of it: the least that one in may have (as the
      // largest of the complements), and the most that one of the others may have
      const float x = of_key(score);
      const float off = margin.of_group(of_key(a), both ? of_key(b) : 0.f);
      const int low = key_of(x - off), high = score == kNone ? kNone : key_of(x + off);
      const int least = ~wave_max(in ? ~low : kNone), next = wave_max(in ? kNone : high);
      if (next != kNone && least <= next) in = in_best_groups<E>(p, l, lanes, lane, lds);
    }
    const uint64_t chosen = __builtin_amdgcn_ballot_w64(in);
    // lane / lanes (the quotient is at least half a 64th from a whole number)
    const int group = (int)((lane + 0.5f) * __builtin_amdgcn_rcpf((float)lanes));
    const int out = (int)(chosen >> (group & 63) & 1) - 1;
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = pick(out, kNone, v[i]);
  }
  int at[E];
#pragma unroll
  for (int i = 0; i < E; ++i) at[i] = lane * E + i;
  sort_down<E>(v, at);
  mine = -1;
  // lane j has the key of choice j; those behind the last are chosen too until one is
  // apart, so that the real choices are among them
  int key = kNone, last = kNone, n = 0;
  bool known = true;
  for (;; ++n) {
    const int best = wave_max(v[0]);
    if (best == kNone) break;
    if (n >= p.top && (!p.bias || margin.apart(of_key(last), of_key(best)))) break;
    known = n < 64;
    if (!known) break;
    last = best;
    const int w = __builtin_ctzll(__builtin_amdgcn_ballot_w64(v[0] == best));
    const int e = __builtin_amdgcn_readlane(at[0], w);
    const int here = -(int)(lane == n), pop = -(int)(lane == w);
    mine = pick(here, e, mine);
    key = pick(here, best, key);
#pragma unroll
    for (int i = 0; i + 1 < E; ++i) {
      v[i] = pick(pop, v[i + 1], v[i]);
      at[i] = pick(pop, at[i + 1], at[i]);
    }
    v[E - 1] = pick(pop, kNone, v[E - 1]);
  }
  if (!known) return false;
  if (p.bias) {
    const int next = __shfl_down(key, 1);
    const bool close = lane + 1 < n && !margin.apart(of_key(key), of_key(next));
    if (__builtin_amdgcn_ballot_w64(close)) {
      // their order in 64 bits
      const Exact<E> exact(p, l);
      double x = -INFINITY;
      if (lane < n) x = exact.biased(fminf(row[mine], FLT_MAX), p.bias[mine]);
      int rank = lane < n ? 0 : lane;
      for (int j = 0; j < n; ++j) {
        const double y = lane_value(x, j);
        const int e = __builtin_amdgcn_readlane(mine, j);
        rank += lane < n && ((y > x) | ((y == x) & (e < mine)));
      }
      mine = __builtin_amdgcn_ds_permute(rank * 4, mine);
    }
  }
  if (lane >= p.top) mine = -1;
  return true;
}

// The choices in 64 bits from the start, the scores in LDS: for groups that share lanes
// and for more than 64 scores too close to each other.
template <int E>
__device__ __forceinline__ int choose(const RouteProblem& p, const float (&l)[E], int lane,
                                      double* v) {
  const Exact<E> exact(p, l);
  float bias[E];
  if (p.bias) load_row<E>(p.bias, p.experts, lane, 0.f, bias);
#pragma unroll
  for (int i = 0; i < E; ++i)   // without a bias the scores have the logits' order
    v[lane * E + i] = p.bias && l[i] > -INFINITY ? exact.biased(l[i], bias[i]) : l[i];
  wave_fence();
  if (p.group_top < p.groups) {
    const int size = p.group_size;
    const bool sums = p.group_best == 2;
    double gs[E];   // of groups lane E + i
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int g = lane * E + i;
      double a = -INFINITY, b = -INFINITY;
      if (g < p.groups)
        for (int k = 0; k < size; ++k) {
          const double x = v[g * size + k];
          if (x > a) {
            b = a;
            a = x;
          } else if (x > b) {
            b = x;
          }
        }
      if (sums && !p.bias) {
        a = a > -INFINITY ? exact.score(a) : a;
        b = b > -INFINITY ? exact.score(b) : b;
      }
      gs[i] = sums && b > -INFINITY ? a + b : a;
    }
    wave_fence();
    uint32_t in = 0;
    for (int j = 0; j < p.group_top; ++j) {
      const int g = wave_best<E>(gs, lane);
      if (g < 0) break;
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (lane * E + i == g) {
          gs[i] = -INFINITY;
          in |= 1u << i;
        }
    }
#pragma unroll 1
    for (int i = 0; i < E; ++i) {
      const int g = lane * E + i;
      if (g < p.groups && !(in >> i & 1))
        for (int k = 0; k < size; ++k) v[g * size + k] = -INFINITY;
    }
    wave_fence();
  }
  int mine = -1;
  for (int j = 0; j < p.top; ++j) {
    double x[1] = {-INFINITY};
    int at = 0;
#pragma unroll 1
    for (int i = 0; i < E; ++i)
      if (v[lane * E + i] > x[0]) {
        x[0] = v[lane * E + i];
        at = i;
      }
    const int w = wave_best<1>(x, lane);
    if (w < 0) break;
    const int e = w * E + __builtin_amdgcn_readlane(at, __builtin_amdgcn_readfirstlane(w));
    if (lane == j) mine = e;
    if (lane == w) v[e] = -INFINITY;
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
  __shared__ double lds[kWaves][64 * (E > 1 ? E : 2)];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t t = (int64_t)tile_id() * kWaves + wave;
  if (t >= p.tokens) return;
  float l[E];
  load_logits<E>(p, t, lane, l);
  int e;
  if (!choose_fast<E>(p, p.logits + t * p.ldl, l, lane, lds[wave], e)) {
    wave_fence();
    e = choose<E>(p, l, lane, lds[wave]);
  }
  const bool there = e >= 0;
  float x = 0.f, w;   // this lane's chosen logit
  if (there) x = fminf(p.logits[t * p.ldl + e], FLT_MAX);
  if (p.sigmoid) {
    w = there ? sigmoid(x) : 0.f;
    if (p.renorm) w = share_of_sigmoid(x, w, there);
  } else if (p.renorm) {
    w = share_of_chosen(x, there);
  } else {
    const float m = largest<E>(l), sum = exp_sum<E>(l, m);
    w = there ? expf(x - m) / sum : 0.f;
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
// Where one share is above a half, the difference at it would have lost the bits that 1 less
// that share has.  With m its place,
//   g_i - sum q_k g_k = (g_i - g_m) + sum q_k (g_m - g_k)
// where m itself adds nothing.
// Lane j forms the gradient of choice j; it is handed to the expert's lane choice
// by choice, so an expert named twice gets both.

// g - sum q_k g_k of the lanes' entries.
__device__ __forceinline__ float centred(float q, float g, bool there) {
  const uint64_t most = __builtin_amdgcn_ballot_w64(there && q > 0.5f);
  if (most == 0) return g - wave_sum(there ? q * g : 0.f);
  const float gm = lane_value(g, __builtin_ctzll(most));
  return (g - gm) + wave_sum(there ? q * (gm - g) : 0.f);
}

template <int E>
__global__ void __launch_bounds__(kThreads) route_grad_kernel(RouteProblem p) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t t = (int64_t)tile_id() * kWaves + wave;
  if (t >= p.tokens) return;
  const float* row = p.logits + t * p.ldl;
  int e = lane < p.top ? p.choice[t * p.top + lane] : -1;
  float x = e >= 0 && e < p.experts ? row[e] : -INFINITY;
  const bool there = x > -INFINITY;
  x = fminf(x, FLT_MAX);
  const float g = there ? p.scale * p.dweight[t * p.top + lane] : 0.f;
  const bool all = !p.sigmoid && !p.renorm;   // every expert has a share
  float mine = g;
  if (!all) {
    // 1 - s is the sigmoid of -x: taken from s it would have no bits left above x = 17
    const float s = p.sigmoid && there ? sigmoid(x) : 0.f, rest = p.sigmoid ? sigmoid(-x) : 1.f;
    if (p.renorm) {
      const float q = p.sigmoid ? share_of_sigmoid(x, s, there) : share_of_chosen(x, there);
      mine = q * centred(q, g, there) * rest;
    } else {
      mine = s * rest * g;
    }
  }
  float d[E];
#pragma unroll
  for (int i = 0; i < E; ++i) d[i] = 0.f;
  for (int j = 0; j < p.top; ++j) {
    const int to = __builtin_amdgcn_readlane(there ? e : -1, j);
    const float y = lane_value(mine, j);
    if (to < 0) continue;
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (lane * E + i == to) d[i] += y;
  }
  if (all) {
    float w[E], sum = 0.f;
    load_logits<E>(p, t, lane, w);
    const float m = largest<E>(w);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      w[i] = w[i] > -INFINITY ? expf(w[i] - m) : 0.f;
      sum += w[i];
    }
    sum = wave_sum(sum);
    // one above a half is alone at m, and alone has w 1: two there have a sum of 2
    const bool leads = sum < 2.f;
    float base = 0.f, add;
    if (leads) {
      base = wave_sum(there && x == m ? g : 0.f);
      float others = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) others += w[i] < 1.f ? w[i] * (base - d[i]) : 0.f;
      add = wave_sum(others) / sum;
    } else {
      add = -wave_sum(there ? expf(x - m) / sum * g : 0.f);
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float by = leads && w[i] == 1.f ? 0.f : d[i] - base;
      d[i] = w[i] > 0.f ? w[i] / sum * (by + add) : 0.f;
    }
  }
  float* out = p.dlogits + t * p.lddl;
  store_row<E>(out, p.experts, lane, d);
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
