// The product of few rows of A with a strip of B's columns, K split over the
// waves of a workgroup (gfx950): bound by reading the weights, or A, once.
//
// Wave w takes the chunks of 16 U k numbered w, w + kWaves, ... and multiplies them
// from registers with v_mfma_f32_16x16x4_f32, whose operand layout needs no
// LDS: lane (h = l / 16, c = l % 16) holds A[row c][k slot h] and B[k slot h][column
// c].  One 16-byte load gives a lane four consecutive k of its row of A (k =
// 4 h + s in step s = 0 .. 3), so B's element of step s is k = 4 h + s too: with B
// stored N x K that is the same 16-byte load of row n; with B stored K x N the
// lane loads NB consecutive columns of row k, so 16 lanes read runs of 64 NB
// bytes and block j multiplies columns n0 + NB c + j.
//
// Multi-dword loads need 4-byte alignment only, so any pitch loads at full
// width; the last k (K % 16) and the last columns are loaded element by element.
#pragma once

#include "grouped_internal.h"
#include "mfma_common.h"

namespace gemmf32 {
namespace grouped {

using namespace mfma;

typedef float floatx4 __attribute__((ext_vector_type(4)));

static __device__ __attribute__((aligned(16))) const float kZeroRow[4] = {0.f, 0.f, 0.f, 0.f};

typedef float floatx4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef float floatx2_a4 __attribute__((ext_vector_type(2), aligned(4)));
// B's loads: non-temporal where B is read once (kOnce)
template <bool kOnce>
__device__ __forceinline__ float4 load_b4(const float* p) {
  if constexpr (!kOnce) return load4(p);
  const floatx4 v = __builtin_nontemporal_load(reinterpret_cast<const floatx4_a4*>(p));
  return make_float4(v.x, v.y, v.z, v.w);
}
template <bool kOnce>
__device__ __forceinline__ float2 load_b2(const float* p) {
  float2 v;
  if constexpr (kOnce) {
    const floatx2_a4 x = __builtin_nontemporal_load(reinterpret_cast<const floatx2_a4*>(p));
    v = make_float2(x.x, x.y);
  } else {
    __builtin_memcpy(&v, p, sizeof(v));
  }
  return v;
}
template <bool kOnce>
__device__ __forceinline__ float load_b1(const float* p) {
  return kOnce ? __builtin_nontemporal_load(p) : *p;
}

// The tile of 16 RM rows by 16 NB columns n0 .. of A B, each wave's share of K
// left in red (kWaves * 16 RM * 16 NB floats of LDS) behind a barrier.  row_at(i): the
// row of A of tile row i, -1 for none.  kTB: B stored N x K; kOnce: its loads are
// non-temporal.
template <int kWaves, int RM, int NB, bool kTB, int U, bool kOnce, class RowAt>
__device__ __forceinline__ void rows_product(float* red, const float* A, int64_t lda, RowAt row_at,
                                             const float* B, int64_t ldb, int N, int n0, int K,
                                             int wave, int lane) {
  const int h = lane >> 4, c = lane & 15;
  // this lane's rows of A; a row that is not there reads zeros
  const float* a_row[RM];
  bool a_in[RM];
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    const int r = row_at(16 * i + c);
    a_in[i] = r >= 0;
    a_row[i] = a_in[i] ? A + (int64_t)r * lda + 4 * h : kZeroRow;
  }
  // this lane's places in B: rows n (stored N x K; those past N read row
  // N - 1, never stored) or columns n0 + NB c .. of row k
  const float* b_row[kTB ? NB : 1];
  int cols = NB;   // of this lane's NB columns, those inside
  if constexpr (kTB) {
#pragma unroll
    for (int j = 0; j < NB; ++j)
      b_row[j] = B + (int64_t)min(n0 + 16 * j + c, N - 1) * ldb + 4 * h;
  } else {
    cols = max(0, min(NB, N - n0 - NB * c));
    b_row[0] = B + (int64_t)(4 * h) * ldb + (cols > 0 ? n0 + NB * c : 0);
  }

  struct Step {   // 16 k
    float4 a[RM];
    float4 b[kTB ? NB : 4];   // stored N x K: .xyzw are k; stored K x N: [s] holds NB columns
  };
  auto load = [&](Step& x, int k) {
#pragma unroll
    for (int i = 0; i < RM; ++i) x.a[i] = load4(a_in[i] ? a_row[i] + k : kZeroRow);
    if constexpr (kTB) {
#pragma unroll
      for (int j = 0; j < NB; ++j) x.b[j] = load_b4<kOnce>(b_row[j] + k);
    } else {
      const float* b = b_row[0] + (int64_t)k * ldb;
      if (cols == NB) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          if constexpr (NB == 4) {
            x.b[s] = load_b4<kOnce>(b + s * ldb);
          } else if constexpr (NB == 2) {
            const float2 v = load_b2<kOnce>(b + s * ldb);
            x.b[s] = make_float4(v.x, v.y, 0.f, 0.f);
          } else {
            x.b[s] = make_float4(load_b1<kOnce>(b + s * ldb), 0.f, 0.f, 0.f);
          }
        }
      } else {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const float* q = b + s * ldb;
          x.b[s] = make_float4(cols > 0 ? q[0] : 0.f, cols > 1 ? q[1] : 0.f,
                               cols > 2 ? q[2] : 0.f, cols > 3 ? q[3] : 0.f);
        }
      }
    }
  };
  // the last K % 16 k, element by element with zeros past K
  auto load_tail = [&](Step& x, int k) {
    const int left = K - k - 4 * h;   // of this lane's four k, those inside
    auto four = [&](const float* q, int64_t step) {
      return make_float4(left > 0 ? q[0] : 0.f, left > 1 ? q[step] : 0.f,
                         left > 2 ? q[2 * step] : 0.f, left > 3 ? q[3 * step] : 0.f);
    };
#pragma unroll
    for (int i = 0; i < RM; ++i)
      x.a[i] = a_in[i] ? four(a_row[i] + k, 1) : make_float4(0.f, 0.f, 0.f, 0.f);
    if constexpr (kTB) {
#pragma unroll
      for (int j = 0; j < NB; ++j) x.b[j] = four(b_row[j] + k, 1);
    } else {
      const float* b = b_row[0] + (int64_t)k * ldb;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const float* q = b + s * ldb;
        const bool in = s < left;
        x.b[s] = make_float4(in && cols > 0 ? q[0] : 0.f, in && cols > 1 ? q[1] : 0.f,
                             in && cols > 2 ? q[2] : 0.f, in && cols > 3 ? q[3] : 0.f);
      }
    }
  };
  floatx4 acc[RM][NB];
#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  auto part = [](const float4& v, int s) { return s == 0 ? v.x : s == 1 ? v.y : s == 2 ? v.z : v.w; };
  auto compute = [&](const Step& x) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
              part(x.a[i], s), kTB ? part(x.b[j], s) : part(x.b[s], j), acc[i][j], 0, 0, 0);
  };

  // whole chunks of 16 U k, two in flight; then whole steps of 16; then the tail
  constexpr int kChunk = 16 * U;
  const int chunks = K / kChunk;
  Step s0[U], s1[U];
  auto load_chunk = [&](Step (&x)[U], int ch) {
#pragma unroll
    for (int u = 0; u < U; ++u) load(x[u], ch * kChunk + 16 * u);
  };
  auto compute_chunk = [&](const Step (&x)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) compute(x[u]);
  };
  if (wave < chunks) {
    load_chunk(s0, wave);
    int ch = wave;
    for (; ch + 2 * kWaves < chunks; ch += 2 * kWaves) {
      load_chunk(s1, ch + kWaves);
      compute_chunk(s0);
      load_chunk(s0, ch + 2 * kWaves);
      compute_chunk(s1);
    }
    if (ch + kWaves < chunks) {
      load_chunk(s1, ch + kWaves);
      compute_chunk(s0);
      compute_chunk(s1);
    } else {
      compute_chunk(s0);
    }
  }
  // what is left, one step of 16 a wave from the last wave down
  const int k_left = chunks * kChunk, steps_left = (K - k_left + 15) / 16;
  const int mine = kWaves - 1 - wave;
  if (mine < steps_left) {
    const int k = k_left + 16 * mine;
    if (k + 16 <= K) {
      load(s0[0], k);
    } else {
      load_tail(s0[0], k);
    }
    compute(s0[0]);
  }

  // ---- the waves' tiles ---------------------------------------------------------
  constexpr int BN = 16 * NB, BM = 16 * RM;
  // a row that is not there: zeros times weights that are not finite were NaN
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    const unsigned there = (unsigned)__ballot(a_in[i]) & 0xffffu;
    if (there != 0xffffu) {
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (!(there >> (4 * h + r) & 1)) acc[i][j][r] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        red[(wave * BM + 16 * i + 4 * h + r) * BN + (kTB ? 16 * j + c : NB * c + j)] = acc[i][j][r];
  __syncthreads();
}

// Element x (row x / BN, column x % BN) of the tile that rows_product left in
// red: the waves' tiles added in wave order.
template <int kWaves, int RM, int NB>
__device__ __forceinline__ float rows_sum(const float* red, int x) {
  float sum = red[x];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) sum += red[w * (16 * RM) * (16 * NB) + x];
  return sum;
}

}  // namespace grouped
}  // namespace gemmf32
