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

namespace gemmf32 {
namespace {

using namespace q4;

// Byte offset of (row r of 16, octet o of 32 k) in a fragment block of 1 KiB:
// rotated by the octet, so that a wave that writes the octets of consecutive rows,
// and one that reads a fragment, both spread over all banks.
__device__ __forceinline__ int fragment(int r, int o) {
  return (((r + 4 * o) & 15) + 16 * o) * 16;
}

template <int BM, int BN, int WM, int WN, bool kE2m1, bool kFold>
struct Tiles {
  static constexpr int kWavesN = BN / WN, kWaves = BM / WM * kWavesN, kThreads = 64 * kWaves;
  static constexpr int kI = WM / 16, kJ = WN / 16;
  static constexpr int kOctets = BM * 4 / kThreads;   // of A, a thread's
  static constexpr int kBytesA = BM * 3 * 64, kBytesW = BN * 64, kBytesS = kFold ? BN * 4 : 0;
  static constexpr int kStage = kBytesA + kBytesW + kBytesS;
  static constexpr int kLds = 2 * kStage + BM * 8;
  static_assert(BM * 4 % kThreads == 0 && BN * 2 <= kThreads && BM <= kThreads, "one share each");

  const Q4Problem& p;
  char* lds;
  int tid, wave, lane, n0;
  const Weights w;
  int64_t K;
  // this thread's share of the loads: octets of A's rows, and 16 codes of a column
  const float* a[kOctets];       // NULL: a row that is not there
  const uint8_t* codes;
  int64_t n;                     // the column whose codes (and scale) it loads
  float x[kOctets][8];
  uint32_t c[2];
  float scale, zero;
  f32x4 acc[kI][kJ];

  __device__ __forceinline__ Tiles(const Q4Problem& p, char* lds, int group, int n0)
      : p(p), lds(lds), tid(threadIdx.x), wave(threadIdx.x >> 6), lane(threadIdx.x & 63), n0(n0),
        w(p, group), K(p.g.K) {}

  // One step's values into registers.
  __device__ __forceinline__ void load(int step) {
    const int64_t k0 = (int64_t)step * 32;
#pragma unroll
    for (int i = 0; i < kOctets; ++i) {
      const int64_t k = k0 + 8 * (tid & 3);
      if (a[i] && k + 8 <= K) {
        __builtin_memcpy(x[i], a[i] + k0, sizeof(x[i]));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i][j] = a[i] && k + j < K ? a[i][k0 + j] : 0.f;
      }
    }
    if (tid < BN * 2) {
      const int64_t k = k0 + 16 * (tid & 1);
      if (k + 16 <= K) {
        __builtin_memcpy(c, codes + k0 / 2, sizeof(c));
      } else {   // bytes behind the row's last are not read
        const int bytes = (int)(K - k + 1) / 2;
        uint64_t v = 0;
        for (int i = 0; i < bytes; ++i) v |= (uint64_t)codes[k0 / 2 + i] << 8 * i;
        c[0] = (uint32_t)v;
        c[1] = (uint32_t)(v >> 32);
      }
      const int64_t at = k0 >> p.group_shift;
      if (step == 0 || at != (k0 - 32) >> p.group_shift) {
        scale = load_scale(w.scale, p.scale_type, w.scale0 + n * p.lds + at);
        if constexpr (!kE2m1) zero = w.zero ? (float)w.zero[n * p.ldz + at] : 8.f;
      }
    }
  }

  // The registers' values into a buffer.
  __device__ __forceinline__ void convert(int buffer) {
    char* to = lds + buffer * kStage;
#pragma unroll
    for (int i = 0; i < kOctets; ++i) {
      const int r = (tid >> 2) + i * (kThreads / 4);
      u32x4 parts[3];
      split8(x[i], parts);
#pragma unroll
      for (int part = 0; part < 3; ++part)
        *reinterpret_cast<u32x4*>(to + ((r >> 4) * 3 + part) * 1024 + fragment(r & 15, tid & 3)) =
            parts[part];
    }
    if (tid < BN * 2) {
      const int col = tid >> 1;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<bf16x8*>(to + kBytesA + (col >> 4) * 1024 +
                                   fragment(col & 15, 2 * (tid & 1) + h)) =
            weights8<kE2m1, !kFold>(c[h], zero, scale);
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
      constexpr int kAtOnce = 2, kGroups = kI * kJ / kAtOnce;
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

  // During step t: the next one's values into the other buffer, and the loads of
  // those behind it.
  __device__ __forceinline__ void refill(int t, int steps) {
    if (t + 1 < steps) convert((t + 1) & 1);
    if (t + 2 < steps) load(t + 2);
  }

  // Places begin .. end - 1, the first BM of them.
  __device__ __forceinline__ void run(const Epilogue& ep, int begin, int end) {
    int* from_row = reinterpret_cast<int*>(lds + 2 * kStage);
    int* to_row = from_row + BM;
    if (tid < BM) {
      const int place = min(begin + tid, end - 1);
      const int r = p.g.ia ? p.g.ia[place] : place, t = p.g.ic ? p.g.ic[place] : place;
      from_row[tid] = r >= 0 && r < p.g.rows_a ? r : -1;
      to_row[tid] = begin + tid < end && t >= 0 && t < p.g.rows_c ? t : -1;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kOctets; ++i) {
      const int r = from_row[(tid >> 2) + i * (kThreads / 4)];
      a[i] = r >= 0 ? p.g.A + r * p.g.lda + 8 * (tid & 3) : nullptr;
    }
    n = min(n0 + (tid >> 1), p.g.N - 1);   // columns past the last are not stored
    codes = w.codes + n * p.ldq + 8 * (tid & 1);
    scale = 1.f;
    zero = 8.f;
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
      for (int j = 0; j < kJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int steps = (int)((K + 31) / 32);
    if (steps > 0) {
      load(0);
      convert(0);
      if (steps > 1) load(1);
      __syncthreads();
      const bool first = wave < kWaves / 2;   // converts first
      for (int t = 0; t < steps; ++t) {
        if (first) refill(t, steps);
        multiply(t & 1);
        if (!first) refill(t, steps);
        __syncthreads();
      }
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

template <int BM, int BN, int WM, int WN, bool kE2m1, bool kFold>
__global__ void __launch_bounds__(64 * (BM / WM) * (BN / WN), BM* BN >= 256 * 256 ? 1 : 2)
    q4_tiles_kernel(Q4Problem p, Epilogue ep, unsigned cap) {
  using T = Tiles<BM, BN, WM, WN, kE2m1, kFold>;
  __shared__ __attribute__((aligned(16))) char lds[T::kLds];
  const int across = (p.g.N + BN - 1) / BN;
  RowTiles tiles{p.g.offsets, p.g.groups, p.g.rows, BM, (int)(threadIdx.x & 63), cap, 0};
  const unsigned total = tiles.total() * (unsigned)across;
  const int id = xcd_position(tile_id(), total);
  if (id < 0) return;
  int group, begin, end;
  unsigned first;
  if (!tiles.find((unsigned)id / across, group, begin, end, first)) return;
  const int at = begin + (int)((unsigned)id / across - first) * BM;
  Epilogue e = ep;
  if (e.bias) e.bias += group * p.g.sbias;
  T tile(p, lds, group, (int)((unsigned)id % across) * BN);
  tile.run(e, at, min(end, at + BM));
}

template <int BM, int BN, int WM, int WN, bool kE2m1, bool kFold>
hipError_t launch(const Q4Problem& p, const Epilogue& e, hipStream_t s) {
  const int64_t rows = most_row_tiles(p.g.rows, p.g.groups, BM);
  const int64_t grid = rows * ((p.g.N + BN - 1) / BN);
  if (grid > INT64_C(0x7fffffff)) return hipErrorInvalidValue;
  q4_tiles_kernel<BM, BN, WM, WN, kE2m1, kFold>
      <<<tile_grid(grid), 64 * (BM / WM) * (BN / WN), 0, s>>>(p, e, (unsigned)rows);
  return hipGetLastError();
}

template <bool kE2m1, bool kFold>
hipError_t by_tile(const Q4Problem& p, const Epilogue& e, hipStream_t s) {
  const int64_t large = ((int64_t)p.g.rows / 256 + p.g.groups / 2) * ((p.g.N + 255) / 256);
  if (large >= 192) return launch<256, 256, 64, 128, kE2m1, kFold>(p, e, s);
  return launch<128, 128, 64, 64, kE2m1, kFold>(p, e, s);
}

}  // namespace

hipError_t launch_q4_tiles(const Q4Problem& p, const Epilogue& e, hipStream_t s) {
  const bool fold = p.scale_type != kScaleE8m0;
  if (p.e2m1) return fold ? by_tile<true, true>(p, e, s) : by_tile<true, false>(p, e, s);
  return fold ? by_tile<false, true>(p, e, s) : by_tile<false, false>(p, e, s);
}

}  // namespace gemmf32
