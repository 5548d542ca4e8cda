// The last step of low-rank adapters beside a shared projection (gfx950): Y[order[i]]
// += H[i] op(U_g) for every place i of adapter g, H places x R.
//
// Bound by reading and writing those rows of Y once.  A wave owns 32 places of one
// adapter by 32 columns: it loads its elements of Y into the accumulators of
// v_mfma_f32_32x32x2_f32 (lane l, register r: row 8 (r / 4) + 4 (l / 32) + r % 4, column
// l % 32), all of them in flight at once, adds the R products, whose operands come
// from registers (lane = (k slot l / 32, row or column l % 32), four consecutive k of a
// row of H to a load), and stores them.  The rank is short, so nothing is worth
// staging in LDS.  A tile has one adapter's rows only: a factor that is not
// finite reaches no other row.  (4095 x 2048, rank 32: 18 us with 32 columns a wave,
// 21 with 64 and more waits for each; 2048 x 1536, rank 8: 6.2, 8.2 and, with 128
// columns, 11.8 us.  Adding the rank as K-tiles of the projection instead saved
// nothing: the sums of each adapter have to be kept apart from the other rows'.)
#include "grouped_internal.h"
#include "mfma_common.h"

namespace gemmf32 {
namespace {

using namespace mfma;

constexpr int kRows = 32, kCols = 32, kWaves = 4;

template <bool kTB>
__global__ void __launch_bounds__(kWaves * 64)
    adapters_add_kernel(AdapterProblem p, int strips, unsigned cap) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 31, lk = lane >> 5;
  RowTiles rt{p.offsets, p.groups, p.places, kRows, lane, cap, 0};
  const unsigned total = rt.total();
  const int id = xcd_position(tile_id(), total * (unsigned)strips);
  if (id < 0) return;
  int g = 0, begin = 0, end = 0;
  unsigned first = 0;
  if (!rt.find((unsigned)id / strips, g, begin, end, first)) return;
  const int i0 = begin + ((int)((unsigned)id / strips) - (int)first) * kRows;
  const int n0 = ((int)((unsigned)id % strips) * kWaves + wave) * kCols;
  if (n0 >= p.N) return;
  // this lane's place, and its row of Y; the rows of its registers come from the
  // lanes that have them
  const int at = i0 + lr;
  int mine = at < end ? p.order[at] : -1;
  if (mine < 0 || mine >= p.M) mine = -1;
  int row[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) row[r] = __shfl(mine, 8 * (r >> 2) + 4 * lk + (r & 3));

  // a row that is not there reads row 0, a column past the last the last: neither
  // is stored
  const int col = min(n0 + lr, p.N - 1);
  floatx16 acc;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[r] = p.Y[max(row[r], 0) * p.ldy + col];

  // k = 8 q + 4 lk + s in step s of group q; places past the end read the last one's H
  const float* h = p.H + (int64_t)min(at, end - 1) * p.ldh + 4 * lk;
  const float* u = p.U + g * p.su + (kTB ? col * p.ldu + 4 * lk : 4 * lk * p.ldu + col);
  const int64_t step = kTB ? 1 : p.ldu;
  auto multiply = [&](const float4& x, const float4& y) {
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(x.x, y.x, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(x.y, y.y, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(x.z, y.z, acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(x.w, y.w, acc, 0, 0, 0);
  };
  for (int k = 0; k + 8 <= p.R; k += 8) {
    const float* q = u + k * step;
    multiply(load4(h + k), kTB ? load4(q) : make_float4(q[0], q[step], q[2 * step], q[3 * step]));
  }
  if (p.R % 8 != 0) {   // the last ones, zeros past the rank
    const int k = p.R / 8 * 8, left = p.R - k - 4 * lk;
    auto some = [&](const float* q, int64_t d) {
      return make_float4(left > 0 ? q[0] : 0.f, left > 1 ? q[d] : 0.f, left > 2 ? q[2 * d] : 0.f,
                         left > 3 ? q[3 * d] : 0.f);
    };
    multiply(some(h + k, 1), some(u + k * step, step));
  }
  if (n0 + lr >= p.N) return;
#pragma unroll
  for (int r = 0; r < 16; ++r)
    if (row[r] >= 0) p.Y[row[r] * p.ldy + col] = acc[r];
}

}  // namespace

hipError_t launch_adapters_add(const AdapterProblem& p, hipStream_t s) {
  const int64_t strips = ((int64_t)p.N + kWaves * kCols - 1) / (kWaves * kCols);
  const int64_t cap = most_row_tiles(p.places, p.groups, kRows);
  if (cap * strips > 0x7fffffff) return hipErrorInvalidConfiguration;
  if (p.trans) {
    hipLaunchKernelGGL((adapters_add_kernel<true>), tile_grid(cap * strips), dim3(kWaves * 64), 0,
                       s, p, (int)strips, (unsigned)cap);
  } else {
    hipLaunchKernelGGL((adapters_add_kernel<false>), tile_grid(cap * strips), dim3(kWaves * 64), 0,
                       s, p, (int)strips, (unsigned)cap);
  }
  return hipGetLastError();
}

}  // namespace gemmf32
