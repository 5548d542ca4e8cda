// The norm of many arrays, sqrt(sum of squares), and the arrays scaled so that it
// is at most a limit.
//
// The arrays are cut into chunks, a workgroup takes every grid-th chunk, and its sum of
// squares goes to the workspace; the next launch adds all of them, each of its
// workgroups alone and in one order, so nothing is counted or waited for and the result
// depends on the sizes only.  Squares are added in 64 bits, which no float's square
// leaves: the sum neither overflows nor loses small arrays beside large ones, and at 8
// bytes of arithmetic for 4 of memory costs nothing beside the read.  Bound by HBM: one
// read for the norm, and a read and a write for the scaled arrays.  264 M floats' norm
// takes 189 us (5.6 TB/s), the norm and the scaled arrays 591 us (5.4 TB/s).
#include "experts_internal.h"

#include <cfloat>

namespace gemmf32 {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kChunk = 16384;   // floats; 4096 were no faster, for 64 arrays of 2.4 M either
constexpr int kAhead = 4;           // loads of 16 bytes that a thread has on the way
constexpr int kArrays = 96;         // of one launch: their table is its argument
constexpr int kMostGroups = 2048;   // workgroups of one launch

// The arrays of one launch: array a's chunks are first[a] .. first[a + 1] - 1.
struct Table {
  const float* x[kArrays];
  float* y[kArrays];
  int64_t n[kArrays];
  int first[kArrays + 1];
  int count;
};

__device__ __forceinline__ int array_of(const Table& t, int chunk) {
  int lo = 0, hi = t.count - 1;   // the last array whose chunks begin at or before it
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Sum over the workgroup; the result in every thread.
__device__ __forceinline__ double group_sum(double x) {
  __shared__ double per_wave[kThreads / 64];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
  if ((threadIdx.x & 63) == 0) per_wave[threadIdx.x >> 6] = x;
  __syncthreads();
  double sum = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) sum += per_wave[w];
  return sum;
}

__device__ __forceinline__ void add_square(double& s, float x) { s += (double)x * (double)x; }

constexpr int kStep = 4 * kThreads;   // floats that the workgroup reads at once
__device__ __forceinline__ float4 load4(const float* x) {
  float4 v;
  __builtin_memcpy(&v, x, sizeof(v));
  return v;
}
// Past the caches, which keep the read arrays instead (120 arrays of 264 M floats: 5 % less
// time than with ordinary stores).
template <class F>
__device__ __forceinline__ void store4(float* y, float4 v, F f) {
  typedef float vector __attribute__((ext_vector_type(4), aligned(4)));
  __builtin_nontemporal_store(vector{f(v.x), f(v.y), f(v.z), f(v.w)},
                              reinterpret_cast<vector*>(y));
}

// y = f(x) for every array (those in place if kInPlace), the last chunks first: they are the
// ones that the caches still hold.
template <bool kInPlace, class F>
__device__ __forceinline__ void map_arrays(const Table& t, F f) {
  for (int c = t.first[t.count] - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
    const int a = array_of(t, c);
    const int64_t from = (c - t.first[a]) * kChunk, to = min(t.n[a], from + kChunk);
    const float* x = t.x[a];
    float* y = t.y[a];
    if (!kInPlace && x == y) continue;
    int64_t i = from + 4 * threadIdx.x;
    for (; i + (kAhead - 1) * kStep + 4 <= to; i += kAhead * kStep) {
      float4 v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) v[k] = load4(x + i + k * kStep);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) store4(y + i + k * kStep, v[k], f);
    }
    for (; i + 4 <= to; i += kStep) store4(y + i, load4(x + i), f);
    for (; i < to; ++i) y[i] = f(x[i]);
  }
}

__global__ void __launch_bounds__(kThreads) norm_parts_kernel(Table t, double* part) {
  double s0 = 0, s1 = 0, s2 = 0, s3 = 0;
  const int chunks = t.first[t.count];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int a = array_of(t, c);
    const int64_t from = (c - t.first[a]) * kChunk, to = min(t.n[a], from + kChunk);
    const float* x = t.x[a];
    int64_t i = from + 4 * threadIdx.x;
    for (; i + (kAhead - 1) * kStep + 4 <= to; i += kAhead * kStep) {
      float4 v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) v[k] = load4(x + i + k * kStep);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        add_square(s0, v[k].x);
        add_square(s1, v[k].y);
        add_square(s2, v[k].z);
        add_square(s3, v[k].w);
      }
    }
    for (; i + 4 <= to; i += kStep) {
      const float4 v = load4(x + i);
      add_square(s0, v.x);
      add_square(s1, v.y);
      add_square(s2, v.z);
      add_square(s3, v.w);
    }
    for (; i < to; ++i) add_square(s0, x[i]);
  }
  const double sum = group_sum((s0 + s1) + (s2 + s3));
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__device__ __forceinline__ double norm_of(const double* part, int parts) {
  double s = 0;
  for (int i = threadIdx.x; i < parts; i += kThreads) s += part[i];
  return sqrt(group_sum(s));
}

__global__ void __launch_bounds__(kThreads)
    norm_join_kernel(const double* part, int parts, float* norm) {
  const double v = norm_of(part, parts);
  if (threadIdx.x == 0) *norm = (float)v;
}

// y = x limit / norm where the norm is finite and above the limit, else y = x.  The factor
// is a float, where that is a normal number; a smaller one would have few bits or none,
// though its products with large elements are ordinary numbers, and stays in 64 bits.
__global__ void __launch_bounds__(kThreads)
    norm_scale_kernel(Table t, const double* part, int parts, float limit, float* norm) {
  const double v = norm_of(part, parts);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)v;
  const double by = (double)limit / v;
  if (!(v > (double)limit && v < (double)INFINITY)) {
    map_arrays<false>(t, [](float x) { return x; });
  } else if (by >= (double)FLT_MIN) {
    const float f = (float)by;
    map_arrays<true>(t, [f](float x) { return x * f; });
  } else {
    map_arrays<true>(t, [by](float x) { return (float)((double)x * by); });
  }
}

// Calls f(table, workgroups) for each launch's share of the arrays, those without
// an element left out.  Chunks of one launch stay below 2^30 (an array has at most
// 2^26): a share also ends before that.
template <class F>
hipError_t for_tables(int64_t count, const float* const* x, const int64_t* n, float* const* out,
                      F f) {
  Table t;
  int64_t i = 0;
  while (i < count) {
    t.count = 0;
    int64_t chunks = 0;
    for (; i < count && t.count < kArrays; ++i) {
      if (n[i] <= 0) continue;
      const int64_t more = (n[i] + kChunk - 1) / kChunk;
      if (chunks + more > INT64_C(1) << 30) break;
      t.x[t.count] = x ? x[i] : nullptr;
      t.y[t.count] = out ? out[i] : const_cast<float*>(t.x[t.count]);   // in place
      t.n[t.count] = n[i];
      t.first[t.count++] = (int)chunks;
      chunks += more;
    }
    if (t.count == 0) break;
    t.first[t.count] = (int)chunks;
    const hipError_t e = f(t, (int)(chunks < kMostGroups ? chunks : kMostGroups));
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t norm_parts(int64_t count, const int64_t* n) {
  // the workgroups of every launch, counted as for_tables launches them
  size_t parts = 0;
  const hipError_t e = for_tables(count, nullptr, n, nullptr, [&](const Table&, int groups) {
    parts += (size_t)groups;
    return hipSuccess;
  });
  return e == hipSuccess ? parts : 0;
}

hipError_t launch_norm(int64_t count, const float* const* x, const int64_t* n, bool clip,
                       float* const* out, float limit, float* norm, double* part, hipStream_t s) {
  int parts = 0;
  hipError_t e = for_tables(count, x, n, nullptr, [&](const Table& t, int groups) {
    norm_parts_kernel<<<groups, kThreads, 0, s>>>(t, part + parts);
    parts += groups;
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  if (!clip || parts == 0) {
    norm_join_kernel<<<1, kThreads, 0, s>>>(part, parts, norm);
    return hipGetLastError();
  }
  return for_tables(count, x, n, out, [&](const Table& t, int groups) {
    norm_scale_kernel<<<groups, kThreads, 0, s>>>(t, part, parts, limit, norm);
    norm = nullptr;   // written once
    return hipGetLastError();
  });
}

}  // namespace gemmf32
