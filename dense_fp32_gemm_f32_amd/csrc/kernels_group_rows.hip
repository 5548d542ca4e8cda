// Rows ordered by group: a stable counting sort of `n` group numbers.
//
// offsets[g] counts the entries below group g; an entry's place is offsets[g]
// plus the number of earlier entries of its group.  One workgroup of 16 waves:
// each wave counts a contiguous share of the entries in LDS counters of its
// own, the counters are turned into first places by a scan over (group, wave),
// and each wave then deals its share out 64 entries at a time, an entry's rank
// among the 64 coming from ballots over the bits of the group number.  Only
// the counts use atomics, and whole numbers add up the same in any order.
#include "grouped_internal.h"

namespace gemmf32 {
namespace {

constexpr int kWaves = 16;

// The lanes whose value equals this lane's in its low `bits` bits (and whose
// `in` is set), by one ballot for each bit.
__device__ __forceinline__ unsigned long long same_lanes(int v, bool in, int bits) {
  unsigned long long m = __ballot(in);
  for (int b = 0; b < bits; ++b) {
    const bool one = (v >> b) & 1;
    const unsigned long long bal = __ballot(in && one);
    m &= one ? bal : ~bal;
  }
  return m;
}

__global__ void __launch_bounds__(kWaves * 64)
    group_rows_kernel(int n, int groups, int bits, int per_row, const int* __restrict__ index,
                      int* __restrict__ offsets, int* __restrict__ order,
                      int* __restrict__ rows) {
  __shared__ int count[kWaves * kMaxGroups];   // [wave][group]
  __shared__ int wave_sum[kWaves];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  for (int i = tid; i < kWaves * groups; i += kWaves * 64) count[i] = 0;
  __syncthreads();

  // a wave's share: whole batches of 64
  const int batches = (int)(((int64_t)n + 63) / 64);
  const int per = (batches + kWaves - 1) / kWaves;
  const int64_t i0 = min((int64_t)n, (int64_t)wave * per * 64);
  const int64_t i1 = min((int64_t)n, i0 + (int64_t)per * 64);
  int* mine = count + wave * groups;
  for (int64_t i = i0 + lane; i < i1; i += 64) {
    const int g = index[i];
    if (g >= 0 && g < groups) atomicAdd(&mine[g], 1);
  }
  __syncthreads();

  // thread g: the first places of group g's share of each wave
  int total = 0;
  if (tid < groups) {
    for (int w = 0; w < kWaves; ++w) {
      const int c = count[w * groups + tid];
      count[w * groups + tid] = total;
      total += c;
    }
  }
  int incl = total;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 63) wave_sum[wave] = incl;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += wave_sum[w];
    all += wave_sum[w];
  }
  const int first = before + incl - total;
  if (tid < groups) {
    offsets[tid] = first;
    for (int w = 0; w < kWaves; ++w) count[w * groups + tid] += first;
  }
  if (tid == 0) offsets[groups] = all;
  __syncthreads();

  for (int64_t base = i0; base < i1; base += 64) {
    const int64_t i = base + lane;
    const int g = i < i1 ? index[i] : -1;
    const bool in = g >= 0 && g < groups;
    const unsigned long long same = same_lanes(g, in, bits);
    if (in) {
      const int rank = __popcll(same & ((1ull << lane) - 1));
      const int at = mine[g] + rank;
      order[at] = (int)i;
      if (rows) rows[at] = (int)i / per_row;
    }
    // the last lane of each group moves the group's place on, after every
    // lane has read it (a wave's LDS accesses keep their order)
    __builtin_amdgcn_wave_barrier();
    if (in && (same >> lane) == 1ull) mine[g] += __popcll(same);
    __builtin_amdgcn_wave_barrier();
  }
  for (int64_t i = (int64_t)all + tid; i < n; i += kWaves * 64) {
    order[i] = -1;
    if (rows) rows[i] = -1;
  }
}

}  // namespace

hipError_t launch_group_rows(int n, int groups, int per_row, const int* index, int* offsets,
                             int* order, int* rows, hipStream_t s) {
  if (n < 0 || groups < 0 || groups > kMaxGroups || per_row < 1) return hipErrorInvalidValue;
  int bits = 0;
  while ((1 << bits) < groups) ++bits;
  hipLaunchKernelGGL(group_rows_kernel, dim3(1), dim3(kWaves * 64), 0, s, n, groups, bits, per_row,
                     index, offsets, order, rows);
  return hipGetLastError();
}

}  // namespace gemmf32
