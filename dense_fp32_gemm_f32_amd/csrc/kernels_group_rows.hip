// Rows ordered by group: a stable counting sort of `n` group numbers, one launch.
//
// offsets[g] counts the entries below group g; an entry's place is offsets[g]
// plus the number of earlier entries of its group.  Each workgroup of 16 waves
// deals out a share of the entries, and counts all entries itself -- those
// before its share, in it (by wave) and behind it -- so that no workgroup waits
// for another and nothing passes through memory.  The counts are turned into
// first places by a scan over the groups, and each wave deals its entries out 64
// at a time, an entry's rank among the 64 coming from ballots over the bits of
// the group number.  Only the counts use atomics (in LDS, four copies against
// conflicts), and whole numbers add up the same in any order.
//
// Bound by launch latency up to some thousand entries, then by the LDS counting
// of all entries in every workgroup (64 to 4096 entries: 9 us with the launch, 65536:
// 12 us against 68 us in one workgroup, 262144: 32 us).
#include "grouped_internal.h"

namespace gemmf32 {
namespace {

constexpr int kWaves = 16, kThreads = kWaves * 64;
constexpr int kCopies = 4;
constexpr int kMaxBlocks = 64;

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

// Adds the entries [from, to) to count[group], all threads.
__device__ __forceinline__ void count_entries(const int* __restrict__ index, int64_t from,
                                              int64_t to, int groups, int* count) {
  constexpr int kAhead = 4;   // 16-byte loads in flight
  int64_t i = from + 4 * (int64_t)threadIdx.x;
  auto add = [&](int g) {
    if (g >= 0 && g < groups) atomicAdd(&count[g], 1);
  };
  for (; i + 4 * (kAhead - 1) * kThreads + 4 <= to; i += 4 * kAhead * kThreads) {
    int v[kAhead][4];
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      __builtin_memcpy(v[a], index + i + 4 * a * kThreads, sizeof(v[a]));
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
#pragma unroll
      for (int k = 0; k < 4; ++k) add(v[a][k]);
  }
  for (; i < to; i += 4 * kThreads)
    for (int k = 0; k < 4 && i + k < to; ++k) add(index[i + k]);
}

__global__ void __launch_bounds__(kThreads)
    group_rows_kernel(int n, int share, int groups, int bits, int per_row,
                      const int* __restrict__ index, int* __restrict__ offsets,
                      int* __restrict__ order, int* __restrict__ rows) {
  __shared__ int before[kCopies * kMaxGroups], behind[kCopies * kMaxGroups];
  __shared__ int count[kWaves * kMaxGroups];   // [wave][group], of this share
  __shared__ int wave_sum[kWaves];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  for (int i = tid; i < kCopies * groups; i += kThreads) before[i] = behind[i] = 0;
  for (int i = tid; i < kWaves * groups; i += kThreads) count[i] = 0;
  __syncthreads();

  // this workgroup's share, and each wave's part of it (whole batches of 64)
  const int64_t s0 = min((int64_t)n, (int64_t)blockIdx.x * share);
  const int64_t s1 = min((int64_t)n, s0 + share);
  const int64_t i0 = min(s1, s0 + (int64_t)wave * (share / kWaves));
  const int64_t i1 = min(s1, i0 + share / kWaves);
  int* mine = count + wave * groups;
  for (int64_t i = i0 + lane; i < i1; i += 64) {
    const int g = index[i];
    if (g >= 0 && g < groups) atomicAdd(&mine[g], 1);
  }
  count_entries(index, 0, s0, groups, before + (wave % kCopies) * groups);
  count_entries(index, s1, n, groups, behind + (wave % kCopies) * groups);
  __syncthreads();

  // thread g: how many of group g come before each wave's part, and in all
  int total = 0, first_here = 0;
  if (tid < groups) {
    for (int c = 0; c < kCopies; ++c) first_here += before[c * groups + tid];
    total = first_here;
    for (int w = 0; w < kWaves; ++w) {
      const int c = count[w * groups + tid];
      count[w * groups + tid] = total;
      total += c;
    }
    for (int c = 0; c < kCopies; ++c) total += behind[c * groups + tid];
  }
  int incl = total;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 63) wave_sum[wave] = incl;
  __syncthreads();
  int below = 0, all = 0;
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) below += wave_sum[w];
    all += wave_sum[w];
  }
  const int first = below + incl - total;
  if (tid < groups) {
    if (blockIdx.x == 0) offsets[tid] = first;
    for (int w = 0; w < kWaves; ++w) count[w * groups + tid] += first;
  }
  if (blockIdx.x == 0 && tid == 0) offsets[groups] = all;
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
  // places of no entry, this workgroup's share of them
  for (int64_t i = max((int64_t)all, s0) + tid; i < s1; i += kThreads) {
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
  // shares of whole batches for every wave, at most kMaxBlocks of them
  int64_t blocks = ((int64_t)n + kThreads - 1) / kThreads;
  blocks = blocks < 1 ? 1 : blocks > kMaxBlocks ? kMaxBlocks : blocks;
  const int64_t share = ((n + blocks - 1) / blocks + kThreads - 1) / kThreads * kThreads;
  hipLaunchKernelGGL(group_rows_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, n,
                     (int)(share > 0 ? share : kThreads), groups, bits, per_row, index, offsets,
                     order, rows);
  return hipGetLastError();
}

}  // namespace gemmf32
