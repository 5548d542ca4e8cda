// Which kernel a grouped product, or the gradient of its weights, takes: rules on
// sizes, pitches and alignment alone.  Host code without a HIP call, apart from the
// kernels so that tests can ask which of them a call reaches.
#pragma once

#include <algorithm>
#include <cstdint>

#include "grouped_internal.h"

namespace gemmf32 {

inline bool on_16_bytes(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// ---- C[ic(i)] = act(alpha s_g A[ia(i)] op(B_g) + beta C[ic(i)] + bias_g) ------------
enum class ProductKernel {
  Rows,           // K split over waves (kernels_grouped_rows.hip)
  Mixed,          // 128 x 128 tiles and 64 x 64 quarters, 16-byte copies
  Even64,         // 64 x 64 tiles, 16-byte copies
  Even64Single,   // 64 x 64 tiles, copies of single floats; B stored K x N only
  Even128Single,  // 128 x 128 tiles, copies of single floats
};

inline ProductKernel product_kernel(const GroupedProblem& p) {
  constexpr int64_t kRound = 256;   // workgroups in a round of the CUs
  // 16-byte copies need whole chunks of both operands inside: bases, pitches
  // and strides of 16 bytes, and the contiguous sizes multiples of 4
  const bool wide = on_16_bytes(p.A) && on_16_bytes(p.B) && p.lda % 4 == 0 && p.ldb % 4 == 0 &&
                    (p.groups == 1 || p.sb % 4 == 0) && p.K % 4 == 0 && (p.tb || p.N % 4 == 0);
  // few rows in a group, few columns, or few sums: bound by one read of B or of A,
  // or by the latency of a tile (16 groups of 32, 1024 x 1024: 27 us against 43 us
  // for the tiles; of 64: 34 against 43; of 96: 49 against 43; 64 groups of 48: 130
  // against 77)
  const int64_t busy = std::min(p.rows, p.groups), sums = (int64_t)p.rows * p.N;
  if (p.N <= 64 || p.rows <= 32 * busy || (p.rows <= 64 * busy && sums <= 1 << 20) ||
      sums <= 1 << 18)
    return ProductKernel::Rows;
  // about how many 128 x 128 and 64 x 64 tiles
  const int64_t tiles =
      ((int64_t)p.rows / 128 + p.groups / 2) * (((int64_t)p.N + 127) / 128);
  const int64_t tiles64 = ((int64_t)p.rows / 64 + p.groups / 2) * (((int64_t)p.N + 63) / 64);
  if (wide) {
    // tiles that leave three CUs in eight idle (2 groups of 512, 4096 x 512: 60 us
    // against 86 us for the tiles; 3 of 512, 1024 x 512, half as many tiles more: 30
    // against 26)
    if (tiles64 <= kRound / 8 * 5) return ProductKernel::Rows;
    // 64 x 64 tiles, four workgroups a CU, below a round of the CUs (21 groups of 261,
    // 1280 x 384: 71 us against 87 us in mixed tiles), where the second round would be
    // neither nearly empty nor full (8 of 512, 1024 x 1280: 111 against 123), and for
    // groups that fill few of the rows of 128 (64 of 128, 512 x 768: 78 against 86)
    const bool small = tiles < kRound || (tiles >= kRound / 4 * 5 && tiles < 2 * kRound) ||
                       p.rows <= 192 * (int64_t)p.groups;
    return small ? ProductKernel::Even64 : ProductKernel::Mixed;
  }
  // copies of single floats.  B stored N x K: below four rounds of 128 x 128 tiles the
  // kernel for few rows, whose 16-byte loads fit any row (3 groups of 500, 1501 x 1001:
  // 56 us against 75 us in 64 x 64 tiles; 16 of 437, 515 x 1027: 92 against 136 in tiles
  // of 128; 4 of 3000, 1027 x 1025: 287 against 338; 2 of 4096, 2047 x 1001: 392
  // against 335; 8 of 2048, 2049 x 2047: 1978 against 1314).  Some shapes below lose up
  // to a quarter; over 215 shapes of 2 to 24 groups the rule is 2 % above the faster
  // of the two on average, and rules by the fill of the last round are no nearer.
  if (p.tb) return tiles < 4 * kRound ? ProductKernel::Rows : ProductKernel::Even128Single;
  // Stored K x N below four rounds of 64 x 64 tiles, where the last round counts for
  // most (13 of 161, 769 x 1001: 61 against 68 us; 16 of 200, 511 x 1025: 58 against
  // 72; 2 of 1300, 1501 x 1001: 112 against 122; 8 of 250, 513 x 1023, two whole rounds:
  // 44 against 37; 8 of 512, 2049 x 1023, four: 235 against 214); then those, and 128 x
  // 128 tiles where they make two rounds (8 x 1000 x 1023 x 2047: 333 us against 452).
  // Over the same 215 shapes 5 % above the fastest of the three on average, by the
  // fill of the last round 5 to 7 %.
  if (tiles64 < 4 * kRound) return ProductKernel::Rows;
  return tiles >= 2 * kRound ? ProductKernel::Even128Single : ProductKernel::Even64Single;
}

// ---- the adapters' shared projection, M x N over K, where its rows are not few --------
// By the grouped product's kernels with one group, else by gemm_f32_fused:
//   - from 192 tiles of 128 x 128 on, where gemm_f32_fused takes those tiles, while the
//     64 x 64 tiles still make three rounds of the CUs or fewer (2048 x 1536 x 1024, three
//     rounds: 59 us against 70; 3000 x 1024 x 2048: 111 against 130; 1792 x 2048 x 1024,
//     four: 76 against 70);
//   - few rows with W stored transposed (100 x 2048 x 2048: 19 us against 37; 128 x
//     1024 x 4096: 25 against 69; 65 x 4096 x 1024, past the limit: 21 against 21).
inline bool projection_grouped(const GroupedProblem& p) {
  const int64_t M = p.rows, N = p.N;
  const bool wide = on_16_bytes(p.A) && on_16_bytes(p.B) && p.lda % 4 == 0 && p.ldb % 4 == 0 &&
                    p.K % 4 == 0 && (p.tb || p.N % 4 == 0);
  auto tiles_of = [&](int64_t side) { return (M + side - 1) / side * ((N + side - 1) / side); };
  return (wide && tiles_of(128) >= 192 && tiles_of(64) <= 3 * 256) ||
         (p.tb && M <= 128 && M * N <= 1 << 18);
}

// ---- C_g = alpha sum_i A[ia(i)]^T B[ib(i)] + beta C_g -------------------------------
// M or N of at most 64: the kernel that reads the wide operand once
// (kernels_grouped_wgrad_thin.hip, which plans its own slices)
inline bool wgrad_thin(const GroupedProblem& p) { return p.M <= 64 || p.N <= 64; }

struct GradientTiles {
  bool large;   // 128 x 128 tiles, else 64 x 64
  bool wide;    // 16-byte copies, else of single floats
  int slices;   // of each group's places
};

inline GradientTiles gradient_tiles(const GroupedProblem& p) {
  auto tiles_of = [&](int side) {
    return ((int64_t)p.M + side - 1) / side * (((int64_t)p.N + side - 1) / side) * p.groups;
  };
  GradientTiles t;
  t.wide = on_16_bytes(p.A) && on_16_bytes(p.B) && p.lda % 4 == 0 && p.ldb % 4 == 0 &&
           p.M % 4 == 0 && p.N % 4 == 0;
  // 128 x 128 tiles, two a CU, where they make two rounds or more (16 groups of
  // 512, 1024 x 1024: 148 us against 168 us for 64 x 64; 1024 x 2048 in 8 uneven
  // groups of 8192 places in all: 289 against 328 us; 1023 x 2047 with single-float
  // copies, 8000 places: 362 against 459 us); below that a tile of a long group
  // would run alone (3000 + 1000, 1024 x 1024: 219 against 108 us)
  t.large = tiles_of(128) >= 512;
  // Below that up to four workgroups of 64 x 64 a CU, by slices of 256 places or more
  // in groups of average size and of 2048 in a group that has nearly all, whose sums
  // go through the workspace and a second launch (2 groups of 2048, 256 x 256: 16 us
  // against 54 us in one slice; 1 of 4096, 768 x 768: 59 against 129; 2 of 2000, 511 x
  // 300, single floats: 40 against 120; 2 of 4096, 1024 x 512: 89 against 132; 8 of 256,
  // 256 x 256, stays in one slice: 11 against 13 for 2).
  const int64_t s =
      t.large ? 1
              : std::min(1024 / tiles_of(64), std::max(p.rows / (256 * (int64_t)p.groups),
                                                       (int64_t)p.rows / 2048));
  t.slices = (int)std::max((int64_t)1, s);
  return t;
}

}  // namespace gemmf32
