// Grouped products with few rows in a group, or few columns (gfx950): bound by
// reading the weights, or A, once.
//
// A workgroup owns 16 or 32 places of one group by 16 NB columns and its 8
// waves split K: wave w takes the chunks of 16 U k numbered w, w + 8, ... and
// multiplies them from registers with v_mfma_f32_16x16x4_f32, whose operand
// layout needs no LDS: lane (h = l / 16, c = l % 16) holds A[row c][k slot h]
// and B[k slot h][column c].  One 16-byte load gives a lane four consecutive k
// of its row of A (k = 4 h + s in step s = 0 .. 3), so B's element of step s is
// k = 4 h + s too: with B stored N x K that is the same 16-byte load of row n;
// with B stored K x N the lane loads NB consecutive columns of row k, so 16
// lanes read runs of 64 NB bytes and block j multiplies columns n0 + NB c + j.
// The waves' partial tiles are added in LDS in wave order.
//
// Multi-dword loads need 4-byte alignment only, so any pitch loads at full
// width; the last k (K % 16) and the last columns are loaded element by element.
#include "grouped_internal.h"
#include "mfma_common.h"

namespace gemmf32 {
namespace {

using namespace mfma;

typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8;
static __device__ __attribute__((aligned(16))) const float kZeros[4] = {0.f, 0.f, 0.f, 0.f};

template <int RM, int NB, bool kTB, int U>
__device__ __forceinline__ void rows_tile(float* red, const GroupedProblem& p, const Epilogue& ep,
                                          int g, int m0, int end, int n0, int wave, int lane) {
  const int h = lane >> 4, c = lane & 15;
  const int N = p.N, K = p.K;
  const float* B = p.B + g * p.sb;
  // this lane's rows of A; a row that is not there reads zeros
  const float* a_row[RM];
  bool a_in[RM];
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    const int at = m0 + 16 * i + c;
    int r = -1;
    if (at < end) {
      r = p.ia ? p.ia[at] : at;
      if (r < 0 || r >= p.rows_a) r = -1;
    }
    a_in[i] = r >= 0;
    a_row[i] = a_in[i] ? p.A + (int64_t)r * p.lda + 4 * h : kZeros;
  }
  // this lane's places in B: rows n (stored N x K; those past N read row
  // N - 1, never stored) or columns n0 + NB c .. of row k
  const float* b_row[kTB ? NB : 1];
  int cols = NB;   // of this lane's NB columns, those inside
  if constexpr (kTB) {
#pragma unroll
    for (int j = 0; j < NB; ++j)
      b_row[j] = B + (int64_t)min(n0 + 16 * j + c, N - 1) * p.ldb + 4 * h;
  } else {
    cols = max(0, min(NB, N - n0 - NB * c));
    b_row[0] = B + (int64_t)(4 * h) * p.ldb + (cols > 0 ? n0 + NB * c : 0);
  }

  struct Step {   // 16 k
    float4 a[RM];
    float4 b[kTB ? NB : 4];   // stored N x K: .xyzw are k; stored K x N: [s] holds NB columns
  };
  auto load = [&](Step& x, int k) {
#pragma unroll
    for (int i = 0; i < RM; ++i) x.a[i] = load4(a_in[i] ? a_row[i] + k : kZeros);
    if constexpr (kTB) {
#pragma unroll
      for (int j = 0; j < NB; ++j) x.b[j] = load4(b_row[j] + k);
    } else {
      const float* b = b_row[0] + (int64_t)k * p.ldb;
      if (cols == NB) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          if constexpr (NB == 4) {
            x.b[s] = load4(b + s * p.ldb);
          } else if constexpr (NB == 2) {
            float2 v;
            __builtin_memcpy(&v, b + s * p.ldb, sizeof(v));
            x.b[s] = make_float4(v.x, v.y, 0.f, 0.f);
          } else {
            x.b[s] = make_float4(b[s * p.ldb], 0.f, 0.f, 0.f);
          }
        }
      } else {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const float* q = b + s * p.ldb;
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
      const float* b = b_row[0] + (int64_t)k * p.ldb;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const float* q = b + s * p.ldb;
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

  // ---- the waves' tiles, added in wave order, and the update ------------------
  constexpr int BN = 16 * NB, BM = 16 * RM, kThreads = kWaves * 64;
#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        red[(wave * BM + 16 * i + 4 * h + r) * BN + (kTB ? 16 * j + c : NB * c + j)] = acc[i][j][r];
  __syncthreads();
  const float scale = p.gscale ? p.gscale[g] : 1.f;
  Epilogue e = ep;
  if (e.bias) e.bias += g * p.sbias;
  for (int x = threadIdx.x; x < BM * BN; x += kThreads) {
    float sum = red[x];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += red[w * BM * BN + x];
    const int at = m0 + x / BN, col = n0 + x % BN;
    if (at >= end || col >= N) continue;
    const int r = p.ic ? p.ic[at] : at;
    if (r < 0 || r >= p.rows_c) continue;
    float* out = p.C + (int64_t)r * p.ldc + col;
    *out = epilogue_apply(e, scale * sum, out, col);
  }
}

template <int NB, bool kTB, int U>
__global__ void __launch_bounds__(kWaves * 64)
    grouped_rows_kernel(GroupedProblem p, Epilogue ep, int strips, unsigned cap) {
  __shared__ float red[kWaves * 32 * 16 * NB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  RowTiles rt{p.offsets, p.groups, p.rows, 32, lane, cap, 0};
  const unsigned total = rt.total();
  const unsigned id = tile_id(), t = id / strips;
  if (t >= total) return;
  int g = 0, begin = 0, end = 0;
  unsigned first = 0;
  if (!rt.find(t, g, begin, end, first)) return;
  const int m0 = begin + (int)(t - first) * 32, n0 = (int)(id % strips) * 16 * NB;
  if (end - m0 <= 16) {
    rows_tile<1, NB, kTB, U>(red, p, ep, g, m0, end, n0, wave, lane);
  } else {
    rows_tile<2, NB, kTB, U>(red, p, ep, g, m0, min(end, m0 + 32), n0, wave, lane);
  }
}

template <int NB, int U>
hipError_t launch(const GroupedProblem& p, const Epilogue& e, hipStream_t s) {
  const int64_t strips = ((int64_t)p.N + 16 * NB - 1) / (16 * NB);
  const int64_t cap = most_row_tiles(p.rows, p.groups, 32);
  if (cap * strips > 0x7fffffff) return hipErrorInvalidConfiguration;
  const dim3 grid = tile_grid(cap * strips), block(kWaves * 64);
  if (p.tb) {
    hipLaunchKernelGGL((grouped_rows_kernel<NB, true, U>), grid, block, 0, s, p, e, (int)strips,
                       (unsigned)cap);
  } else {
    hipLaunchKernelGGL((grouped_rows_kernel<NB, false, U>), grid, block, 0, s, p, e, (int)strips,
                       (unsigned)cap);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_rows(const GroupedProblem& p, const Epilogue& e, hipStream_t s) {
  if (p.N <= 16) return launch<1, 4>(p, e, s);
  if (p.N <= 32 || p.tb) return launch<2, 4>(p, e, s);
  return launch<4, 2>(p, e, s);
}

}  // namespace gemmf32
