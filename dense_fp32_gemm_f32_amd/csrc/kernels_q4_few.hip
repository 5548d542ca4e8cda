// Products with 4-bit weights for few rows: tiles of up to 10 rows by 16 CT columns,
// K split over the 8 waves of a workgroup.  Bound by the read of the codes.
//
// The rows' three bf16 parts are the rows of the matrix instruction: row r's part
// p is row 3 r + p, so that up to 5 rows of A take one instruction for 16 columns
// by 32 k, up to 10 two.  The workgroup splits them once, into LDS
// in the order of the fragments; each wave then takes every 8th chunk of 128 k of
// the workgroup's columns, 16 bytes of codes a lane, and the waves' sums are added
// in LDS in one order.
#include "q4_common.h"

namespace gemmf32 {
namespace {

using namespace q4;

constexpr int kWaves = 8, kThreads = kWaves * 64;
constexpr int kRows = 10;            // rows of a tile, at most
constexpr int kChunkK = 128;         // k of a chunk: four steps of 32
// chunks whose parts are in LDS at once, by matrix instructions a step: at most
// 64 KiB, so that two workgroups share a CU
template <int RT>
constexpr int kPass = 16 / RT;
constexpr int kLdsBytes = 16 * 4 * 1024;

// Fragments of a step of 32 k: RT KiB; row q of the instruction's 16 and octet o of
// the k are 16 bytes, rotated by the step and octet so that the threads that write
// octets of one row spread over the banks.
__device__ __forceinline__ int slot(int q, int octet, int step) {
  return ((q + 4 * octet + step) & 15) + 16 * octet;
}

template <int CT, int NS>
struct Item {   // a wave's chunk of its columns
  u32x4 codes[CT];
  uint32_t scale[CT][NS], zero[CT][NS];   // as they are stored
};

// kRest: the chunk that passes the end of K, of which nothing behind a row's end is
// read.  In whole chunks no branch leaves a load out and nothing looks at what is
// loaded: they stay in flight while the chunk before is multiplied.
template <int CT, bool kE2m1, int NS, bool kRest>
__device__ __forceinline__ void fetch(const Q4Problem& p, const Weights& w, int chunk, int n0,
                                      int lane, Item<CT, NS>& it) {
  const int64_t K = p.g.K, k0 = (int64_t)chunk * kChunkK;
#pragma unroll
  for (int c = 0; c < CT; ++c) {
    // columns past the last read the last row: their sums are not stored
    const int64_t n = min(n0 + 16 * c + (lane & 15), p.g.N - 1);
    const uint8_t* row = w.codes + n * p.ldq;
    if constexpr (kRest)
      it.codes[c] = last_codes(row, k0 + 32 * (lane >> 4), K);
    else
      __builtin_memcpy(&it.codes[c], row + k0 / 2 + 16 * (lane >> 4), sizeof(u32x4));
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int64_t at = (kRest ? min(k0 + 32 * i, K - 1) : k0 + 32 * i) >> p.group_shift;
      it.scale[c][i] = load_scale(w.scale, p.scale_type, w.scale0 + n * p.lds + at);
      if constexpr (!kE2m1) it.zero[c][i] = w.zero ? w.zero[n * p.ldz + at] : 8;
    }
  }
}

// One chunk of a wave: parts are those of its first step in LDS.
template <int RT, int CT, bool kE2m1, int NS>
__device__ __forceinline__ void multiply(const Q4Problem& p, const Item<CT, NS>& it, int step0,
                                         const char* lds, int lane, f32x4 (&acc)[RT][CT]) {
  u32x4 steps[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) steps[c] = by_steps(it.codes[c]);
  f32x4 sum[RT][CT];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    bf16x8 a[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
      a[t] = *reinterpret_cast<const bf16x8*>(
          lds + (((step0 + i) * RT + t) * 64 + slot(lane & 15, lane >> 4, step0 + i)) * 16);
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int s = NS == 1 ? 0 : i;
      const bf16x8 b = weights8<kE2m1, false>(steps[c][i], kE2m1 ? 0.f : (float)it.zero[c][s], 1.f);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const f32x4 none = {0.f, 0.f, 0.f, 0.f};
        sum[t][c] = mfma16(a[t], b, NS == 1 && i > 0 ? sum[t][c] : none);
      }
    }
    if (NS == 4 || i == 3) {
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const float scale = scale_value(it.scale[c][NS == 1 ? 0 : i], p.scale_type);
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[t][c] += sum[t][c] * scale;
      }
    }
    __builtin_amdgcn_sched_barrier(0);   // else all steps' weights are converted first
  }
}

// One tile of `rows` rows, places first .. first + rows - 1.
template <int RT, int CT, bool kE2m1, int NS>
__device__ void tile(const Q4Problem& p, const Epilogue& ep, const Weights& w, int group,
                     int first, int rows, int n0, char* lds, int* row_of) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int64_t K = p.g.K;
  const int chunks = (int)((K + kChunkK - 1) / kChunkK);
  if (tid < rows) {
    const int place = first + tid;
    const int r = p.g.ia ? p.g.ia[place] : place;
    row_of[tid] = r >= 0 && r < p.g.rows_a ? r : -1;
  }
  f32x4 acc[RT][CT];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[t][c] = f32x4{0.f, 0.f, 0.f, 0.f};

  // whole chunks; a part of one behind them is the wave's whose turn it would be
  const int whole = (int)(K / kChunkK);
  // chunks on the way into registers: as many as a wave has in a pass
  constexpr int kAhead = 1;
  Item<CT, NS> ahead[kAhead];
  int chunk = wave;
  if (whole > 0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      fetch<CT, kE2m1, NS, false>(p, w, min(chunk + i * kWaves, whole - 1), n0, lane, ahead[i]);
  }
  const unsigned inverse = (65536 + rows - 1) / rows;   // u / rows for u below 65536 / 16
  for (int base = 0; base < chunks; base += kPass<RT>) {
    const int here = min(kPass<RT>, chunks - base);
    __syncthreads();   // row_of is there; the parts of the pass before are used
    for (int u = tid; u < rows * here * (kChunkK / 8); u += kThreads) {
      const int octet = (int)((unsigned)u * inverse >> 16), r = u - octet * rows;
      const int64_t k = (int64_t)base * kChunkK + 8 * octet;
      const int row = row_of[r];
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
      if (row >= 0) {
        const float* a = p.g.A + row * p.g.lda + k;
        if (k + 8 <= K) {
          __builtin_memcpy(x, a, sizeof(x));
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (k + i < K) x[i] = a[i];
        }
      }
      u32x4 parts[3];
      split8(x, parts);
      const int step = octet >> 2;
#pragma unroll
      for (int part = 0; part < 3; ++part) {
        const int q = 3 * r + part;
        *reinterpret_cast<u32x4*>(lds + ((step * RT + (q >> 4)) * 64 +
                                         slot(q & 15, octet & 3, step)) * 16) = parts[part];
      }
    }
    __syncthreads();
    const int to = min(base + here, whole);
    while (chunk < to) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (chunk >= to) break;
        multiply<RT, CT, kE2m1, NS>(p, ahead[i], (chunk - base) * 4, lds, lane, acc);
        fetch<CT, kE2m1, NS, false>(p, w, min(chunk + kAhead * kWaves, whole - 1), n0, lane,
                                    ahead[i]);
        chunk += kWaves;
      }
    }
    if (whole < chunks && base + here == chunks && wave == whole % kWaves) {
      Item<CT, NS> rest;
      fetch<CT, kE2m1, NS, true>(p, w, whole, n0, lane, rest);
      multiply<RT, CT, kE2m1, NS>(p, rest, (whole - base) * 4, lds, lane, acc);
    }
  }
  __syncthreads();
  // the waves' sums: [wave][row of the instruction][column]
  float* red = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        red[((wave * RT + t) * 16 + 4 * (lane >> 4) + r) * (16 * CT) + 16 * c + (lane & 15)] =
            acc[t][c][r];
  __syncthreads();
  Epilogue e = ep;
  if (e.bias) e.bias += group * p.g.sbias;
  for (int u = tid; u < rows * 16 * CT; u += kThreads) {
    const int r = u / (16 * CT), n = u % (16 * CT);
    float v = 0.f;
    for (int wv = 0; wv < kWaves; ++wv)
#pragma unroll
      for (int part = 0; part < 3; ++part) {
        v += red[((wv * RT * 16) + 3 * r + part) * (16 * CT) + n];
      }
    const int place = first + r;
    const int to = p.g.ic ? p.g.ic[place] : place;
    if (n0 + n < p.g.N && to >= 0 && to < p.g.rows_c) {
      float* c = p.g.C + to * p.g.ldc + n0 + n;
      *c = epilogue_apply(e, row_of[r] >= 0 ? v : 0.f, c, n0 + n);
    }
  }
  __syncthreads();
}

template <int CT, bool kE2m1, int NS>
__global__ void __launch_bounds__(kThreads, 4) q4_few_kernel(Q4Problem p, Epilogue ep) {
  __shared__ __attribute__((aligned(16))) char lds[kLdsBytes];
  __shared__ int row_of[kRows];
  const int group = blockIdx.y;
  int begin, end;
  group_span(p.g.offsets, group, p.g.rows, begin, end);
  const Weights w(p, group);
  // row tiles of one size, along the grid's z and, where there are more, in turn
  const int tiles = (end - begin + kRows - 1) / kRows;
  const int each = tiles > 0 ? (end - begin + tiles - 1) / tiles : 0;
  for (int64_t n0 = (int64_t)blockIdx.x * 16 * CT; n0 < p.g.N; n0 += (int64_t)gridDim.x * 16 * CT)
    for (int i = blockIdx.z; i < tiles; i += gridDim.z) {
      const int first = begin + i * each, rows = min(each, end - first);
      if (rows <= 0) break;
      if (rows <= 5)
        tile<1, CT, kE2m1, NS>(p, ep, w, group, first, rows, (int)n0, lds, row_of);
      else
        tile<2, CT, kE2m1, NS>(p, ep, w, group, first, rows, (int)n0, lds, row_of);
    }
}

template <int CT, bool kE2m1>
hipError_t launch(const Q4Problem& p, const Epilogue& e, hipStream_t s) {
  const int tiles = p.g.offsets ? 1 : (p.g.rows + kRows - 1) / kRows;
  const int strips = (p.g.N + 16 * CT - 1) / (16 * CT);
  const dim3 grid((unsigned)(strips < kGridX ? strips : kGridX), (unsigned)p.g.groups,
                  (unsigned)(tiles < 1024 ? tiles : 1024));
  if (p.group_shift >= 7)
    q4_few_kernel<CT, kE2m1, 1><<<grid, kThreads, 0, s>>>(p, e);
  else
    q4_few_kernel<CT, kE2m1, 4><<<grid, kThreads, 0, s>>>(p, e);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_q4_few(const Q4Problem& p, const Epilogue& e, hipStream_t s) {
  return p.e2m1 ? launch<2, true>(p, e, s) : launch<2, false>(p, e, s);
}

}  // namespace gemmf32
