// Products with 4-bit weights by tiles of many rows.  Bound by the bf16 matrix
// instruction at three products for each of the fp32 one.
//
// K goes in steps of 32, one group of weights at most, two LDS buffers, one
// barrier a step.  A step's operands lie in LDS as the fragments of the 16 x 16 x
// 32 instruction, 16 bytes a lane: A as its three bf16 parts, W without its scale.
// While a step is multiplied, the threads split and convert the next one's values,
// which they have in registers, and load those behind it.  Half of the waves
// convert first and multiply then, the others the other way round, so that on each
// SIMD one wave's vector instructions run beside the other's matrix instructions.
//
// A step's sums are formed without the scale and added to the tile's, times the
// column's scale.  A scale that is a power of two is put into the weights instead,
// which stay bf16 values exactly, and the sums go straight on.
#include "q4_common.h"
#include "q4_routes.h"
#include <type_traits>

namespace gemmf32 {
namespace {

using namespace q4;

// Byte offset of (row r of 16, octet o of 32 k) in a fragment block of 1 KiB: the rows
// exchanged by the octet, so that a wave's write of the octets of consecutive rows
// spreads over all banks (13 cycles of the CU against 32), and its read of a fragment
// takes no longer than one in order (6.3 cycles; with the rows rotated by 4 o: 8, and 16).
__device__ __forceinline__ int fragment(int r, int o) { return ((r ^ 2 * o) + 16 * o) * 16; }

// D: steps whose values are on the way into registers.
// KS: groups of waves, each with every KS-th step and buffers of its own; the first
// adds the others' sums to its own in order.
template <int BM, int BN, int WM, int WN, int KS, int D, int kForm, bool kFold>
struct Tiles {
  static constexpr int kWavesN = BN / WN, kWaves = BM / WM * kWavesN, kThreads = 64 * kWaves;
  static constexpr int kBM = BM, kBN = BN, kAllThreads = KS * kThreads;
  static constexpr int kI = WM / 16, kJ = WN / 16;
  static constexpr int kOctets = BM * 4 / kThreads;   // of A, a thread's
  static constexpr int kBytesA = BM * 3 * 64, kBytesW = BN * 64, kBytesS = kFold ? BN * 4 : 0;
  static constexpr int kStage = kBytesA + kBytesW + kBytesS;
  static constexpr int kSums = KS > 1 ? BM * BN * 4 : 0;
  static constexpr int kBuffers = 2 * kStage > kSums ? 2 * kStage : kSums;
  static constexpr int kLds = KS * kBuffers + BM * 8;
  static_assert(BM * 4 % kThreads == 0 && BN * 2 <= kThreads && BM <= kThreads, "one share each");

  const Q4Problem& p;
  char* lds;         // of this thread's group
  int* rows;         // from_row and to_row of all
  int part_k, tid, wave, lane, n0;   // its group, and its place in that
  const Weights w;
  int64_t K;
  // this thread's share of the loads: octets of A's rows, and 16 codes of a column
  const float* a[kOctets];
  const uint8_t *codes, *zeros;
  int64_t n;                     // the column whose codes (and scale) it loads
  struct Values {
    float x[kOctets][8];
    uint32_t c[2];
    // as they are stored (bytes as bytes: widened here, they would be masked, and so
    // waited for, at the end of the loop that loads them)
    std::conditional_t<kFold, uint32_t, uint8_t> scale;
    uint8_t zero;
  } v[D];
  f32x4 acc[kI][kJ];

  __device__ __forceinline__ Tiles(const Q4Problem& p, char* lds, int group, int n0)
      : p(p), rows(reinterpret_cast<int*>(lds + KS * kBuffers)),
        part_k(KS > 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / kThreads) : 0),
        tid((int)threadIdx.x - part_k * kThreads), wave(tid >> 6), lane(tid & 63), n0(n0),
        w(p, group), K(p.g.K) {
    this->lds = lds + part_k * kBuffers;
  }

  // The values of one of its group's whole steps into registers.  No branch leaves a
  // load out and nothing looks at what is loaded, so that the loads of the steps
  // behind stay in flight when one step's are waited for.
  __device__ __forceinline__ void load(Values& v, int step) {
    const int64_t k0 = ((int64_t)step * KS + part_k) * 32;
#pragma unroll
    for (int i = 0; i < kOctets; ++i) __builtin_memcpy(v.x[i], a[i] + k0, sizeof(v.x[i]));
    __builtin_memcpy(v.c, codes + k0 / 2, sizeof(v.c));
    load_scales(v, k0);
  }
  __device__ __forceinline__ void load_scales(Values& v, int64_t k0) {
    const int64_t at = k0 >> p.group_shift;
    const int64_t i = w.scale0 + n * p.lds + at;
    if constexpr (kFold)
      v.scale = p.scale_type == kScaleF32 ? static_cast<const uint32_t*>(w.scale)[i]
                                          : static_cast<const uint16_t*>(w.scale)[i];
    else
      v.scale = static_cast<const uint8_t*>(w.scale)[i];
    if constexpr (kForm == kIntZeros) v.zero = zeros[at];
  }

  // The same for the part of K behind the whole steps: k past the end reads the last
  // one, and settle_rest() then makes A's values there zeros, as it does the scale of a step
  // that is all behind K (an infinite one times its sum, 0, would be NaN).
  __device__ __forceinline__ void load_rest(Values& v, int step) {
    const int64_t k0 = ((int64_t)step * KS + part_k) * 32, ka = k0 + 8 * (tid & 3),
                  kw = k0 + 16 * (tid & 1);
#pragma unroll
    for (int i = 0; i < kOctets; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v.x[i][j] = a[i][min(ka + j, K - 1) - 8 * (tid & 3)];
    uint8_t bytes[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) bytes[i] = codes[min(kw + 2 * i, K - 1) / 2 - 8 * (tid & 1)];
    __builtin_memcpy(v.c, bytes, sizeof(v.c));
    load_scales(v, min(k0, K - 1));
  }
  __device__ __forceinline__ void settle_rest(Values& v, int step) {
    const int64_t k0 = ((int64_t)step * KS + part_k) * 32, ka = k0 + 8 * (tid & 3);
#pragma unroll
    for (int i = 0; i < kOctets; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (ka + j >= K) v.x[i][j] = 0.f;
    if constexpr (kFold) {
      if (KS > 1 && k0 >= K) v.scale = 0;
    } else {
      // weights with their scale: codes behind K (half a byte that may hold anything, and
      // copies) get the code of weight 0, as one that passes the largest float times 0 is
      // NaN.  (A zero point above 15 has none: then 15 is nearest, and each real code's
      // weight at least as large.)
      const uint32_t none =
          0x11111111u * (kForm == kE2m1 ? 0u : kForm == kInt8 ? 8u : min((uint32_t)v.zero, 15u));
      const int64_t left = K - (k0 + 16 * (tid & 1));   // real ones of this thread's 16
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int n = (int)max((int64_t)0, min(left - 8 * h, (int64_t)8));
        const uint32_t keep = n < 8 ? (1u << 4 * n) - 1u : ~0u;
        v.c[h] = (v.c[h] & keep) | (none & ~keep);
      }
    }
  }

  // The registers' values into a buffer.
  __device__ __forceinline__ void convert(const Values& v, int buffer) {
    char* to = lds + buffer * kStage;
#pragma unroll
    for (int i = 0; i < kOctets; ++i) {
      const int r = (tid >> 2) + i * (kThreads / 4);
      u32x4 parts[3];
      split8(v.x[i], parts);
#pragma unroll
      for (int part = 0; part < 3; ++part)
        *reinterpret_cast<u32x4*>(to + ((r >> 4) * 3 + part) * 1024 + fragment(r & 15, tid & 3)) =
            parts[part];
    }
    if (BN * 2 == kThreads || tid < BN * 2) {
      const int col = tid >> 1;
      const float scale = scale_value(v.scale, kFold ? p.scale_type : kScaleE8m0);
      const float zero = kForm == kIntZeros ? (float)v.zero : 8.f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<bf16x8*>(to + kBytesA + (col >> 4) * 1024 +
                                   fragment(col & 15, 2 * (tid & 1) + h)) =
            weights8<kForm, !kFold>(v.c[h], zero, scale);
      if constexpr (kFold)
        if ((tid & 1) == 0) reinterpret_cast<float*>(to + kBytesA + kBytesW)[col] = scale;
    }
  }

  __device__ __forceinline__ void multiply(int buffer) {
    const char* from = lds + buffer * kStage;
    const int wm = wave / kWavesN, wn = wave % kWavesN, at = fragment(lane & 15, lane >> 4);
    const char* fa = from + wm * kI * 3 * 1024 + at;
    const char* fw = from + kBytesA + wn * kJ * 1024 + at;
    bf16x8 b[kJ];
#pragma unroll
    for (int j = 0; j < kJ; ++j) b[j] = *reinterpret_cast<const bf16x8*>(fw + j * 1024);
    float s[kJ];
    if constexpr (kFold) {
      const float* fs = reinterpret_cast<const float*>(from + kBytesA + kBytesW);
#pragma unroll
      for (int j = 0; j < kJ; ++j) s[j] = fs[wn * WN + 16 * j + (lane & 15)];
    }
    if constexpr (kFold) {
      // two blocks' sums are formed while the two before them are folded in.  The
      // compiler, left alone, moves the folds behind the refill, whose branches end the
      // block, and holds (or spills) all sums until then: the empty asm statements want
      // each fold's result where it is.
      constexpr int kAtOnce = kJ % 2 ? 1 : 2, kGroups = kI * kJ / kAtOnce;
      f32x4 sum[2][kAtOnce];
      bf16x8 part[3];
#pragma unroll
      for (int g = 0; g <= kGroups; ++g) {
        const int i = g * kAtOnce / kJ, j0 = g * kAtOnce % kJ;
        if (g < kGroups) {
          if (j0 == 0) {
#pragma unroll
            for (int q = 0; q < 3; ++q)
              part[q] = *reinterpret_cast<const bf16x8*>(fa + (i * 3 + q) * 1024);
          }
#pragma unroll
          for (int q = 0; q < 3; ++q)
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
              const f32x4 none = {0.f, 0.f, 0.f, 0.f};
              sum[g & 1][j] = mfma16(part[q], b[j0 + j], q ? sum[g & 1][j] : none);
            }
        }
        if (g > 0) {
          const int fi = (g - 1) * kAtOnce / kJ, fj = (g - 1) * kAtOnce % kJ;
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[fi][fj + j][r] = fmaf(sum[(g - 1) & 1][j][r], s[fj + j], acc[fi][fj + j][r]);
            asm volatile("" : "+v"(acc[fi][fj + j]));
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kI; ++i) {
        bf16x8 part[3];
#pragma unroll
        for (int q = 0; q < 3; ++q)
          part[q] = *reinterpret_cast<const bf16x8*>(fa + (i * 3 + q) * 1024);
#pragma unroll
        for (int q = 0; q < 3; ++q)
#pragma unroll
          for (int j = 0; j < kJ; ++j) acc[i][j] = mfma16(part[q], b[j], acc[i][j]);
      }
    }
  }

  // Places begin .. end - 1, the first BM of them.
  __device__ __forceinline__ void run(const Epilogue& ep, int begin, int end) {
    int* from_row = rows;
    int* to_row = rows + BM;
    if (part_k == 0 && tid < BM) {
      const int place = min(begin + tid, end - 1);
      const int r = p.g.ia ? p.g.ia[place] : place, t = p.g.ic ? p.g.ic[place] : place;
      from_row[tid] = r >= 0 && r < p.g.rows_a ? r : -1;
      to_row[tid] = begin + tid < end && t >= 0 && t < p.g.rows_c ? t : -1;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kOctets; ++i) {
      const int r = from_row[(tid >> 2) + i * (kThreads / 4)];
      // a row that is not there reads the first one; its sums are not used
      a[i] = p.g.A + max(r, 0) * p.g.lda + 8 * (tid & 3);
    }
    // columns past the last are not stored; threads without a column load one too
    n = min(n0 + (tid >> 1) % BN, p.g.N - 1);
    codes = w.codes + n * p.ldq + 8 * (tid & 1);
    if constexpr (kForm == kIntZeros) zeros = w.zero + n * p.ldz;
    // whole steps of each group; none where A has no row at all
    const int steps = p.g.rows_a > 0 ? (int)(K / (32 * KS)) : 0;
    // Waves w and w + 4 share a SIMD.  One of them refills before it multiplies: its
    // refill of a step stands behind the barrier of the step before, so that all waves
    // run one loop and no path through it leaves loads out.
    const int first = (__builtin_amdgcn_readfirstlane(threadIdx.x) >> 8 & 1) ^ 1;
    const int last = steps - 1;
    // what is left of K; its loads go out before all others where there are registers
    const bool rest = p.g.rows_a > 0 && K % (32 * KS) != 0;
    Values behind;
    if (D > 1 && rest) load_rest(behind, steps);
    if (steps > 0) {
      Values v0, v1;
      load(v0, 0);
      load(v1, min(1, last));
#pragma unroll
      for (int d = 1; d <= D; ++d) load(v[d % D], min(d + first, last));
      convert(v0, 0);
      if (first) convert(v1, 1);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
      for (int j = 0; j < kJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (steps > 0) {
      for (int t = 0;;) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
          multiply(t & 1);
          if (first) __syncthreads();
          // the step behind the next one of this wave (past the last, that one again,
          // which nobody reads) into its buffer, and the loads of the one D further
          Values& next = v[(d + 1) % D];
          convert(next, (t + first + 1) & 1);
          load(next, min(t + first + 1 + D, last));
          if (!first) __syncthreads();
          if (++t == steps) goto done;   // (a break would lead back to the loop's head)
        }
      }
    done:
      __syncthreads();
    }
    if (rest) {
      if constexpr (D == 1) load_rest(v[0], steps);
      settle_rest(D > 1 ? behind : v[0], steps);
      convert(D > 1 ? behind : v[0], 0);
      __syncthreads();
      multiply(0);
      __syncthreads();
    }
    if constexpr (KS > 1) {
      // (the last step's barrier is behind all reads of the buffers)
      constexpr int kVec = kI * kJ;
      f32x4* sums = reinterpret_cast<f32x4*>(lds) + wave * kVec * 64 + lane;
      if (part_k > 0) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) sums[i * 64] = acc[i / kJ][i % kJ];
      }
      __syncthreads();
      if (part_k > 0) return;
      for (int g = 1; g < KS; ++g)
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          acc[i / kJ][i % kJ] += *reinterpret_cast<f32x4*>(reinterpret_cast<char*>(sums + i * 64) +
                                                           g * kBuffers);
    }
    const int wm = wave / kWavesN, wn = wave % kWavesN;
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = wm * WM + 16 * i + 4 * (lane >> 4) + r;
        const int to = to_row[row];
        const bool there = from_row[row] >= 0;
        if (to >= 0) {
          float* out = p.g.C + to * p.g.ldc;
#pragma unroll
          for (int j = 0; j < kJ; ++j) {
            const int col = n0 + wn * WN + 16 * j + (lane & 15);
            if (col < p.g.N)
              out[col] = epilogue_apply(ep, there ? acc[i][j][r] : 0.f, out + col, col);
          }
        }
      }
  }
};

template <class T>
__global__ void __launch_bounds__(T::kAllThreads, T::kLds > 80 * 1024 ? 1 : 2)
    q4_tiles_kernel(Q4Problem p, Epilogue ep, unsigned cap) {
  __shared__ __attribute__((aligned(16))) char lds[T::kLds];
  const int across = (p.g.N + T::kBN - 1) / T::kBN;
  RowTiles tiles{p.g.offsets, p.g.groups, p.g.rows, T::kBM, (int)(threadIdx.x & 63), cap, 0};
  const unsigned total = tiles.total() * (unsigned)across;
  const int id = xcd_position(tile_id(), total);
  if (id < 0) return;
  int group, begin, end;
  unsigned first;
  if (!tiles.find((unsigned)id / across, group, begin, end, first)) return;
  const int at = begin + (int)((unsigned)id / across - first) * T::kBM;
  Epilogue e = ep;
  if (e.bias) e.bias += group * p.g.sbias;
  T tile(p, lds, group, (int)((unsigned)id % across) * T::kBN);
  tile.run(e, at, min(end, at + T::kBM));
}

template <class T>
hipError_t launch(const Q4Problem& p, const Epilogue& e, hipStream_t s) {
  const int64_t rows = most_row_tiles(p.g.rows, p.g.groups, T::kBM);
  const int64_t grid = rows * ((p.g.N + T::kBN - 1) / T::kBN);
  if (grid > INT64_C(0x7fffffff)) return hipErrorInvalidValue;
  q4_tiles_kernel<T><<<tile_grid(grid), T::kAllThreads, 0, s>>>(p, e, (unsigned)rows);
  return hipGetLastError();
}

template <int kForm, bool kFold>
hipError_t by_tile(const Q4Problem& p, const Epilogue& e, hipStream_t s) {
  switch (q4_tile(p)) {
    case kTile256: return launch<Tiles<256, 256, 64, 128, 1, 1, kForm, kFold>>(p, e, s);
    case kTile256x192: return launch<Tiles<256, 192, 64, 96, 1, 1, kForm, kFold>>(p, e, s);
    case kTile256x128: return launch<Tiles<256, 128, 64, 64, 1, 1, kForm, kFold>>(p, e, s);
    case kTile128: return launch<Tiles<128, 128, 64, 64, 2, 1, kForm, kFold>>(p, e, s);
    case kTile64x128: return launch<Tiles<64, 128, 32, 64, 2, 2, kForm, kFold>>(p, e, s);
    case kTile64: return launch<Tiles<64, 64, 32, 32, 4, 2, kForm, kFold>>(p, e, s);
    case kTile32x64: return launch<Tiles<32, 64, 32, 32, 4, 4, kForm, kFold>>(p, e, s);
    default: return launch<Tiles<32, 32, 32, 32, 8, 2, kForm, kFold>>(p, e, s);
  }
}

}  // namespace

hipError_t launch_q4_tiles(const Q4Problem& p, const Epilogue& e, hipStream_t s) {
  const bool fold = p.scale_type != kScaleE8m0;
  if (p.e2m1) return fold ? by_tile<kE2m1, true>(p, e, s) : by_tile<kE2m1, false>(p, e, s);
  if (p.zero)
    return fold ? by_tile<kIntZeros, true>(p, e, s) : by_tile<kIntZeros, false>(p, e, s);
  return fold ? by_tile<kInt8, true>(p, e, s) : by_tile<kInt8, false>(p, e, s);
}

}  // namespace gemmf32
