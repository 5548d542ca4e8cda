// One output tile of a grouped product on the CDNA4 matrix cores, its K-tiles
// copied straight from global memory into LDS (gfx950).
//
// The tiles, LDS layouts, swizzles, fragments and the order of copies, reads and
// MFMAs are those of the extended-operation kernel (kernels_mfma_ex_dma.hip):
// operand "KC" has k contiguous and lies in LDS as [r][k] with swizzled 16-byte
// chunks, operand "RC" has its rows r contiguous and lies as [k][r]; two LDS
// buffers, one barrier for each K-tile.  What differs:
//
//   - the rows of a KC operand, or the k of an RC operand, may be gathered
//     through an index;
//   - k past the end, and gathered k whose index is outside either matrix, are
//     copied from a block of zeros in global memory, so K needs no padding and no
//     value outside is ever read.  Rows that are not there read row 0 and columns
//     past the last read column 0: they reach only sums that are not stored, or,
//     for a row whose index is outside, are stored as the zeros they count as;
//   - a lane copies V floats at once: 4 where both operands allow it, else 1,
//     which any pitch and alignment does.
#pragma once

#include <cstdint>
#include <type_traits>

#include "grouped_internal.h"
#include "mfma_common.h"

namespace gemmf32 {
namespace grouped {

using namespace mfma;

// What copies of absent values read.
static __device__ __attribute__((aligned(16))) const float kZeros[4] = {0.f, 0.f, 0.f, 0.f};

// Lane l copies V floats from g into LDS at lds_wave + V l.  The address of
// LDS comes from M0, saved and restored around the copy, which needs one wait
// state behind the write (s_nop); written as inline assembly so that the
// kernel's own waits alone order copies and reads.  (load_lds16, which leaves
// M0 to the compiler, makes the 64 x 64 tiles slower: 4096 x 1280 x 1024 in one
// group, N x K: 94 against 99 us.)
template <int V>
__device__ __forceinline__ void copy_to_lds(const float* g, float* lds_wave) {
  static_assert(V == 1 || V == 4, "copies of 4 or 16 bytes");
  const uint32_t lds_addr = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds_wave);
  uint32_t saved;
  if constexpr (V == 4) {
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dwordx4 %1, off\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "v"(g), "s"(lds_addr)
        : "memory");
  } else {
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %2\n\t"
        "s_nop 0\n\t"
        "global_load_lds_dword %1, off\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "v"(g), "s"(lds_addr)
        : "memory");
  }
}

// The rows an operand is gathered by: row i of the operand is row at(i) of the
// matrix, -1 where there is none.
struct Gather {
  const int* index;   // NULL: the identity
  int limit;          // rows of the matrix
  __device__ __forceinline__ int at(int i, int end) const {
    if (i >= end) return -1;
    const int r = index ? index[i] : i;
    return r >= 0 && r < limit ? r : -1;
  }
};

// One operand's K-tile: R rows by BK, copied by kWaves waves, V floats a lane.
// kGatherK: k itself is gathered (an RC operand whose k are places).
template <int R, int BK, int kWaves, bool KC, int V, bool kGatherK = false>
struct Operand {
  static_assert(!(KC && kGatherK), "gathered k needs the rows contiguous");
  static constexpr int kLds = R * BK;
  static constexpr int kCopyWaves = kWaves;
  static constexpr bool kGathered = kGatherK;
  static constexpr int kCopies = R * BK / V / (kWaves * 64);   // copies a lane makes
  static_assert(R * BK % (V * kWaves * 64) == 0, "copies divide evenly over the threads");
  static_assert(KC || R % 64 == 0, "the [k][r] swizzle needs 64-wide rows");

  const float* src[kCopies];   // this lane's place of each copy at k = 0
  int row[kGatherK ? kCopies : 1];   // gathered k: the index entry of the next K-tile's copy

  // (r, k) of the first of the V floats at LDS float `f`
  __device__ __forceinline__ static void logical(int f, int& r, int& k) {
    if constexpr (KC) {
      r = f / BK;
      const int p = f % BK;
      k = 4 * ((p >> 2) ^ swz_a<BK / 4>(r)) + (p & 3);
    } else {
      k = f / R;
      r = (f % R) ^ swz_b(k);
    }
  }
  __device__ __forceinline__ static int k_of(int v, int wave, int lane) {
    int r, k;
    logical(((v * kWaves + wave) * 64 + lane) * V, r, k);
    return k;
  }
  // KC with gathered rows: row_at(r) is the matrix row of tile row r
  template <class RowAt>
  __device__ __forceinline__ void init_kc(const float* base, int64_t ld, int wave, int lane,
                                          RowAt row_at) {
#pragma unroll
    for (int v = 0; v < kCopies; ++v) {
      int r, k;
      logical(((v * kWaves + wave) * 64 + lane) * V, r, k);
      src[v] = base + (int64_t)row_at(r) * ld + k;
    }
  }
  // RC: columns r0 + r of a matrix with `cols` columns, row k at k * ld
  __device__ __forceinline__ void init_rc(const float* base, int64_t ld, int r0, int cols,
                                          int wave, int lane) {
#pragma unroll
    for (int v = 0; v < kCopies; ++v) {
      int r, k;
      logical(((v * kWaves + wave) * 64 + lane) * V, r, k);
      src[v] = base + (r < cols - r0 ? r0 + r : 0) + (kGatherK ? 0 : (int64_t)k * ld);
    }
  }
  // gathered k: fetch the index entries of the K-tile at k0 (places first + k;
  // past the end, the last place's).  They are looked at by copy() only: a use
  // here would wait for them, and so for the copies in flight.
  __device__ __forceinline__ void fetch_rows(const Gather& ga, int first, int k0, int k_end,
                                             int wave, int lane) {
    if constexpr (kGatherK) {
      if (ga.index) {
#pragma unroll
        for (int v = 0; v < kCopies; ++v)
          row[v] = ga.index[first + max(0, min(k0 + k_of(v, wave, lane), k_end - 1))];
      } else {
#pragma unroll
        for (int v = 0; v < kCopies; ++v) row[v] = first + k0 + k_of(v, wave, lane);
      }
    }
  }
  // in (gathered k): this k is inside and has a row in both operands
  __device__ __forceinline__ void copy(int v, float* lds, int64_t ld, int k0, int k_end, bool in,
                                       int wave, int lane) const {
    const float* g;
    if constexpr (kGatherK) {
      g = in ? src[v] + (int64_t)row[v] * ld : kZeros;
    } else {
      g = src[v] + (KC ? (int64_t)k0 : (int64_t)k0 * ld);
      // only the last K-tile can be part full
      if (k0 + BK > k_end) g = k_of(v, wave, lane) < k_end - k0 ? g : kZeros;
    }
    copy_to_lds<V>(g, lds + (v * kWaves + wave) * (64 * V));
  }

  // Fragment reads of k group q (8 k), as in the extended-operation kernel.
  static constexpr int units(int frags) { return KC ? frags : 2 * frags; }
  template <int kFrag>
  __device__ __forceinline__ static void read(float (&f)[4][kFrag], const float* lds, int wr,
                                              int lr, int lk, int q, int unit) {
    if constexpr (KC) {
      const int r = wr + 32 * unit + lr;
      const float4 x =
          *reinterpret_cast<const float4*>(&lds[r * BK + 4 * ((2 * q + lk) ^ swz_a<BK / 4>(r))]);
      f[0][unit] = x.x;
      f[1][unit] = x.y;
      f[2][unit] = x.z;
      f[3][unit] = x.w;
    } else {
      const int i = unit / 2, s0 = 2 * (unit % 2);
      const int col = (wr + 32 * i + lr) ^ (lk << 5);
      f[s0][i] = lds[(8 * q + 4 * lk + s0) * R + col];
      f[s0 + 1][i] = lds[(8 * q + 4 * lk + s0 + 1) * R + col];
    }
  }
};

// Where the K loop's copies come from: two operands over k in [0, k_end), whole
// K-tiles but for the last; one K-tile of zeros where k_end is 0.  seek(t) points
// the copies at K-tile t, or at the last one, for t = 0, 1, 2, ... in turn.
// Where k is gathered the index has an entry at `first`.
template <int BK, class OpA_, class OpB_>
struct Source {
  using OpA = OpA_;
  using OpB = OpB_;
  static constexpr int kWaves = OpA::kCopyWaves;
  static_assert(kWaves == OpB::kCopyWaves, "the same waves copy both operands");
  OpA a;
  OpB b;
  int64_t lda, ldb;
  int k_end, wave, lane;
  Gather ga{nullptr, 0}, gb{nullptr, 0};
  int first = 0;
  int k0 = 0;

  __device__ __forceinline__ Source(int64_t lda_, int64_t ldb_, int k_end_, int wave_, int lane_)
      : lda(lda_), ldb(ldb_), k_end(k_end_), wave(wave_), lane(lane_) {}
  __device__ __forceinline__ int tiles() const { return max(1, (k_end + BK - 1) / BK); }
  __device__ __forceinline__ void seek(int t) {
    k0 = min(t, tiles() - 1) * BK;
    a.fetch_rows(ga, first, k0, k_end, wave, lane);
    b.fetch_rows(gb, first, k0, k_end, wave, lane);
  }
  // Copies of a K-tile go out in order of idx.  Both operands gathered along k: a
  // place whose row is outside either matrix is zeros in both, so that it adds
  // nothing, whatever stands opposite.  Copy v of either operand has the same k, so
  // one test serves both (1023 x 2047 over 8000 places: 350 us; with each operand's
  // copy testing both rows 368, each its own row only 355).
  bool in[OpA::kGathered ? OpA::kCopies : 1];
  __device__ __forceinline__ void copy(float* la, float* lb, int idx) {
    const int v = idx < OpA::kCopies ? idx : idx - OpA::kCopies;
    if constexpr (OpA::kGathered) {
      static_assert(std::is_same<OpA, OpB>::value, "the operands' copies are alike");
      if (idx < OpA::kCopies)
        in[v] = OpA::k_of(v, wave, lane) < k_end - k0 && (unsigned)a.row[v] < (unsigned)ga.limit &&
                (unsigned)b.row[v] < (unsigned)gb.limit;
    }
    bool there = true;
    if constexpr (OpA::kGathered) there = in[v];
    if (idx < OpA::kCopies) {
      a.copy(v, la, lda, k0, k_end, there, wave, lane);
    } else {
      b.copy(v, lb, ldb, k0, k_end, there, wave, lane);
    }
  }
};

// The K loop of a BM x BN tile, wave tiles WM x WN, over src's K-tiles.  src may
// copy with more waves than the tile has: those beyond only copy.  kNoSpare: no
// copies past the last K-tile, a branch around each copy instead.  (The gradient
// of 40 weights of 513 x 257 over 7 places each, one K-tile: 20 us against 24 us; of 8
// of 1024 x 2048 over 1024: 291 against 294; but the rows' gradient 2048 x 1024: 300
// against 293.)
// pool: 2 (BM + BN) BK floats of LDS, read by no wave any more.
template <int BM, int BN, int BK, int WM, int WN, bool kNoSpare = false, class Src>
__device__ __forceinline__ void k_loop(float* pool, Src& src, int wave, int lane,
                                       floatx16 (&acc)[WM / 32][WN / 32]) {
  using OpA = typename Src::OpA;
  using OpB = typename Src::OpB;
  constexpr int kWavesM = BM / WM;
  constexpr int kFragM = WM / 32, kFragN = WN / 32;
  static_assert(WM % 32 == 0 && WN % 32 == 0 && BM % WM == 0 && BN % WN == 0, "32x32 blocks");
  static_assert(BK % 16 == 0, "an even number of 8-k groups in a K-tile");
  float* const lds_a0 = pool;
  float* const lds_a1 = lds_a0 + OpA::kLds;
  float* const lds_b0 = lds_a1 + OpA::kLds;
  float* const lds_b1 = lds_b0 + OpB::kLds;
  constexpr int kTileCopies = OpA::kCopies + OpB::kCopies;
  const int wr_a = (wave % kWavesM) * WM, wr_b = (wave / kWavesM) * WN;
  const int lr = lane & 31, lk = lane >> 5;
  struct Frag {
    float a[4][kFragM];
    float b[4][kFragN];
  };
  constexpr int kUnitsA = OpA::units(kFragM), kUnitsB = OpB::units(kFragN);
  constexpr int kReadsPerGroup = kUnitsA + kUnitsB;
  auto read_one = [&](Frag& f, const float* la, const float* lb, int q, int idx) {
    if (idx < kUnitsA) {
      OpA::template read<kFragM>(f.a, la, wr_a, lr, lk, q, idx);
    } else {
      OpB::template read<kFragN>(f.b, lb, wr_b, lr, lk, q, idx - kUnitsA);
    }
  };
#pragma unroll
  for (int i = 0; i < kFragM; ++i)
#pragma unroll
    for (int j = 0; j < kFragN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  // one block per wave: odd k-steps go to a second accumulator, added after
  // the loop (a fixed order: even steps + odd steps)
  constexpr bool kDual = kFragM * kFragN == 1;
  floatx16 acc_odd = {};
  auto mfma_one = [&](const Frag& f, int idx) {
    const int s = idx / (kFragM * kFragN);
    const int i = (idx / kFragN) % kFragM, j = idx % kFragN;
    if constexpr (kDual) {
      if (s & 1) {
        acc_odd = __builtin_amdgcn_mfma_f32_32x32x2f32(f.a[s][i], f.b[s][j], acc_odd, 0, 0, 0);
        return;
      }
    }
    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(f.a[s][i], f.b[s][j], acc[i][j], 0, 0, 0);
  };

  constexpr int kGroups = BK / 8;
  constexpr int kMfmaPerGroup = 4 * kFragM * kFragN;
  constexpr int kHalf = kMfmaPerGroup / 2;
  constexpr int kReadsPerMfma = (kReadsPerGroup + kMfmaPerGroup - 1) / kMfmaPerGroup;
  constexpr int kReadsPer = (kReadsPerGroup + kHalf - 1) / kHalf;
  constexpr int kCopiesPer = (kTileCopies + kHalf - 1) / kHalf;

  const int ktiles = src.tiles();
  if constexpr (Src::kWaves > kWavesM * (BN / WN)) {
    if (wave >= kWavesM * (BN / WN)) {   // the same copies and barriers as below
      src.seek(0);
#pragma unroll
      for (int idx = 0; idx < kTileCopies; ++idx) src.copy(lds_a0, lds_b0, idx);
      src.seek(1);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
#pragma unroll
      for (int idx = 0; idx < kTileCopies; ++idx) src.copy(lds_a1, lds_b1, idx);
      for (int t = 0; t < ktiles; ++t) {
        src.seek(t + 2);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
#pragma unroll
        for (int idx = 0; idx < kTileCopies; ++idx)
          src.copy(t & 1 ? lds_a1 : lds_a0, t & 1 ? lds_b1 : lds_b0, idx);
      }
      __builtin_amdgcn_s_waitcnt(0);
      return;
    }
  }
  // One form of step for all: the copies of a K-tile past the end (where there are
  // any) re-read the last one into the buffer no longer needed; the last step reads
  // fragments it does not use.
  auto copied = [&](int t) { return !kNoSpare || t < ktiles; };
  Frag f0, f1;
  src.seek(0);
#pragma unroll
  for (int idx = 0; idx < kTileCopies; ++idx) src.copy(lds_a0, lds_b0, idx);
  if (copied(1)) src.seek(1);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
#pragma unroll
  for (int idx = 0; idx < kReadsPerGroup; ++idx) read_one(f0, lds_a0, lds_b0, 0, idx);
  if (copied(1)) {
#pragma unroll
    for (int idx = 0; idx < kTileCopies; ++idx) src.copy(lds_a1, lds_b1, idx);
  }

  auto step = [&](int t, auto cur_tag) {
    constexpr int kCur = decltype(cur_tag)::value;
    float* la = kCur ? lds_a1 : lds_a0;
    float* lb = kCur ? lds_b1 : lds_b0;
    float* la_next = kCur ? lds_a0 : lds_a1;
    float* lb_next = kCur ? lds_b0 : lds_b1;
    const bool more = copied(t + 2);
    if (more) src.seek(t + 2);
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      Frag& fc = (q & 1) ? f1 : f0;
      Frag& fn = (q & 1) ? f0 : f1;
      if (q < kGroups - 1) {
#pragma unroll
        for (int i = 0; i < kMfmaPerGroup; ++i) {
          mfma_one(fc, i);
#pragma unroll
          for (int r = 0; r < kReadsPerMfma; ++r)
            if (i * kReadsPerMfma + r < kReadsPerGroup)
              read_one(fn, la, lb, q + 1, i * kReadsPerMfma + r);
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kHalf; ++i) mfma_one(fc, i);
        __builtin_amdgcn_sched_barrier(0);
        // the next K-tile is in LDS and every wave is done with this one
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
          mfma_one(fc, kHalf + i);
#pragma unroll
          for (int r = 0; r < kReadsPer; ++r)
            if (i * kReadsPer + r < kReadsPerGroup)
              read_one(fn, la_next, lb_next, 0, i * kReadsPer + r);
#pragma unroll
          for (int l = 0; l < kCopiesPer; ++l)
            if (i * kCopiesPer + l < kTileCopies && more) src.copy(la, lb, i * kCopiesPer + l);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  };
  for (int t = 0; t < ktiles; t += 2) {
    step(t, std::integral_constant<int, 0>{});
    if (t + 1 < ktiles) step(t + 1, std::integral_constant<int, 1>{});
  }
  // no copy into LDS may still be in flight when the pool is used again
  __builtin_amdgcn_s_waitcnt(0);
  if constexpr (kDual) acc[0][0] += acc_odd;
}

// Mixed tiles: 128 x 128 for whole rounds of the CUs; what is left over, if it
// fills at most three quarters of a round or there is no whole round, as 64 x 64
// quarters of its tiles.  (Grouped product of 8192 x 1024 x 2048 in 8 uneven groups,
// 4.25 rounds: 281 us, against 334 us with 128 x 128 tiles only and 319 us with 64 x
// 64 tiles only; in even groups, four whole rounds, 261, 263 and 296 us.)  The grid
// has a workgroup for every tile and 3 kCus more.
constexpr unsigned kCus = 256;

struct MixedTile {
  bool any, quarter;
  int tm, tn, m_off, n_off;   // the 128 x 128 tile, and the quarter's place in it
};
__device__ __forceinline__ MixedTile mixed_tile(unsigned tiles_m, int tiles_n) {
  const unsigned tiles = tiles_m * (unsigned)tiles_n, over = tiles % kCus;
  const unsigned split = tiles < kCus || over <= kCus / 4 * 3 ? over : 0, whole = tiles - split;
  // (whole is a multiple of the XCDs wherever there are quarters)
  const unsigned id = tile_id();
  MixedTile t{};
  t.quarter = id >= whole;
  const int pos = t.quarter ? xcd_position(id - whole, 4 * split) : xcd_position(id, whole);
  t.any = pos >= 0;
  if (!t.any) return t;
  tile_coords(t.quarter ? (int)whole + pos / 4 : pos, (int)tiles_m, tiles_n, t.tm, t.tn);
  if (t.quarter) {
    t.m_off = (pos & 1) * 64;
    t.n_off = ((pos >> 1) & 1) * 64;
  }
  return t;
}

// The update of a wave's blocks, rows of C through row_c (LDS; -1: not
// written).  One path for the plain product, one that does not read C, one
// that does: a wait for a load also waits for the stores before it, so C's old
// values are loaded a block at a time, and not at all where beta is 0 (the same
// loop with the load under a condition took 27 us more at 8192 x 1024 x 2048).
template <int KFM, int KFN>
__device__ __forceinline__ void store_rows(const floatx16 (&acc)[KFM][KFN], float* C, int64_t ldc,
                                           int N, const Epilogue& ep, float scale,
                                           const int* row_c, int row0, int col0, int lane) {
  const int lr = lane & 31, lk = lane >> 5;
  const bool direct = scale == 1.f && ep.alpha == 1.f && ep.beta == 0.f && !ep.bias && ep.act == 0;
  float bias[KFN];
#pragma unroll
  for (int j = 0; j < KFN; ++j) {
    const int col = col0 + 32 * j + lr;
    bias[j] = ep.bias && col < N ? ep.bias[col] : 0.f;
  }
  // every element: f(its column's bias, its sum, a pointer to it)
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < KFM; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int c = row_c[row0 + 32 * i + 4 * lk + 8 * (r >> 2) + (r & 3)];
        if (c < 0) continue;
        float* const out = C + c * ldc + col0 + lr;
#pragma unroll
        for (int j = 0; j < KFN; ++j)
          if (col0 + 32 * j + lr < N) f(j, acc[i][j][r], out + 32 * j);
      }
  };
  if (direct) {
    each([&](int, float s, float* out) { *out = s; });
  } else if (ep.beta == 0.f) {
    const float alpha = ep.alpha;
    const bool relu = ep.act == 1;
    each([&](int j, float s, float* out) {
      float v = alpha * (scale * s);
      if (ep.bias) v = v + bias[j];
      *out = relu && v < 0.f ? 0.f : v;
    });
  } else {
#pragma unroll
    for (int i = 0; i < KFM; ++i)
#pragma unroll
      for (int j = 0; j < KFN; ++j) {
        const int col = col0 + 32 * j + lr;
        if (col >= N) continue;
        float old[16];
        int row[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          row[r] = row_c[row0 + 32 * i + 4 * lk + 8 * (r >> 2) + (r & 3)];
          // an absent row reads the first element of C, which is there
          old[r] = C[max(row[r], 0) * ldc + col];
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          float v = ep.alpha * (scale * acc[i][j][r]) + ep.beta * old[r];
          if (ep.bias) v = v + bias[j];
          if (ep.act == 1 && v < 0.f) v = 0.f;
          if (row[r] >= 0) C[row[r] * ldc + col] = v;
        }
      }
  }
}

}  // namespace grouped
}  // namespace gemmf32
