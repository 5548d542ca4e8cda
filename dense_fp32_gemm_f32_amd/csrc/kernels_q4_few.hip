// Products with 4-bit weights for few rows (q4_routes.h) and at least 128 k: tiles of up
// to 20 rows.  Bound by the conversion of the codes (95 vector instructions for 2048 of
// them) beside their read: one row of 8192 x 8192 with fp16 scales and zero points takes 18
// us (2.0 TB/s), one of 28672 x 8192, whose codes the caches do not hold, 53, and without
// zero points 41 (2.9 TB/s), where loads alone in the same order take 33.
//
// The rows' three bf16 parts are rows of the matrix instruction: a row has four of its
// 16, of which the last is not used, so that a lane gets the sums of one row's parts and
// adds them by itself; 4 rows of A take one instruction for 16 columns by 32 k.  (With
// all 16 in use, 5 rows and a third, the sums went through LDS whole, three times as
// many.)  A workgroup splits its rows once, into LDS, and goes through strips
// of columns with them (rows whose parts do not fit take K in passes, for each strip
// anew).  A wave takes 16 columns and every kw-th chunk of 128 k, 16 bytes of codes a
// lane; the kw waves of a strip add their sums through LDS in one order, and the 16 / kw
// others have the strips beside it.  Each wave has the codes and scales of its next two
// chunks on the way into registers, whichever strip they are of (four chunks were no
// faster, nor were two chunks of one line of codes in turn).  With 8 waves a workgroup
// the row of 8192 x 8192 took 3 us more, as fewer loads are on the way.
#include "q4_common.h"
#include "q4_routes.h"

#include <algorithm>
#include <type_traits>

namespace gemmf32 {
namespace {

using namespace q4;

constexpr int kWavesLog2 = kQ4FewWavesLog2, kWaves = 1 << kWavesLog2, kThreads = kWaves * 64;
constexpr int kChunkK = 128;         // k of a chunk: four steps of 32
constexpr int kAhead = 2;            // chunks on the way
constexpr int kRowsT = 4;            // rows of an instruction
// the waves' sums (of rt instructions, 4 bytes a lane; two buffers, so that a strip takes
// one barrier, where that leaves the parts room), then the parts; one workgroup to a CU
constexpr int kLdsBytes = 158 * 1024;
constexpr int buffers(int rt) { return rt <= 2 ? 2 : 1; }
constexpr int sum_bytes(int rt) { return buffers(rt) * rt * kThreads * 4; }

// kScales: scales of a chunk (1 for groups of 128 and more), of kBytes bytes each.
template <int kScales, int kBytes>
struct Item {
  u32x4 codes;
  uint32_t scale[(kScales * kBytes + 3) / 4], zero;
};

// a chunk for every wave along K
constexpr int chunks_in_lds(int rt, int rows) {
  return (kLdsBytes - sum_bytes(rt)) / (3 * rows * 256);
}
static_assert(chunks_in_lds(3, kQ4FewRowsDeep) >= kWaves &&
              chunks_in_lds(5, kQ4FewRows) >= kWaves / 2, "room for parts");
static_assert(kQ4FewRowsDeep == 3 * kRowsT && kQ4FewRows == 5 * kRowsT, "as launched");
static_assert(kWaves == 1 << kQ4FewWavesLog2 && kChunkK == kQ4FewK, "as the rules count them");

template <int RT, int kForm, int kScales, int kType>
struct Few {
  static constexpr int kBytes = kType == kScaleF32 ? 4 : kType == kScaleE8m0 ? 1 : 2;
  using It = Item<kScales, kBytes>;
  const Q4Problem& p;
  const Weights w;
  const int64_t K;
  const int row_bytes, along, chunks;   // of a row: bytes of codes, scales, chunks
  const int tid, wave, lane;
  int kw_log2, kwave, side;            // waves along K; this one's place there, and its strip's
  int rows, R;                         // of the tile, and of parts
  int pass;                            // chunks whose parts are in LDS at once
  char *lds, *parts;
  const char* own[RT];   // this lane's parts of the first step
  int *row_of, *row_to;   // rows of A and C, -1: none

  __device__ __forceinline__ Few(const Q4Problem& p, int group, char* lds, int* row_of)
      : p(p), w(p, group), K(p.g.K), row_bytes((int)(((int64_t)p.g.K + 1) / 2)),
        along((int)(((int64_t)p.g.K - 1) >> p.group_shift) + 1),
        chunks((int)(((int64_t)p.g.K + kChunkK - 1) / kChunkK)),
        tid(threadIdx.x), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)),
        lane(threadIdx.x & 63), lds(lds), parts(lds + sum_bytes(RT)), row_of(row_of),
        row_to(row_of + kQ4FewRows) {
    kw_log2 = q4_waves_along_k(p);
    kwave = wave & ((1 << kw_log2) - 1);
    side = wave >> kw_log2;
  }

  // Where a lane's column of a strip begins: its codes, scales and zero points.
  struct Row {
    const uint8_t *codes, *zero;
    const char* scale;
  };
  __device__ __forceinline__ Row row(int strip) const {
    // columns past the last read the last row: their sums are not stored
    const int64_t n =
        min((((int64_t)strip << (kWavesLog2 - kw_log2)) + side) * 16 + (lane & 15),
            (int64_t)p.g.N - 1);
    Row r;
    r.codes = w.codes + n * p.ldq;
    r.scale = static_cast<const char*>(w.scale) + (w.scale0 + n * p.lds) * kBytes;
    if constexpr (kForm == kIntZeros) r.zero = w.zero + n * p.ldz;
    return r;
  }

  // A chunk into registers.  No branch leaves a load out and nothing looks at what is
  // loaded: it stays in flight while others are multiplied.  Where the row ends inside
  // the chunk, its last 16 bytes (and last scales) are read, and moved into place by
  // multiply().
  __device__ __forceinline__ void fetch(It& it, const Row& r, int chunk) const {
    chunk = min(chunk, chunks - 1);
    const int at = min(chunk * (kChunkK / 32) >> (p.group_shift - 5), along - kScales);
    __builtin_memcpy(&it.codes, r.codes + min(chunk * (kChunkK / 2) + 16 * (lane >> 4),
                                              row_bytes - 16), sizeof(u32x4));
    __builtin_memcpy(it.scale, r.scale + (int64_t)at * kBytes, kScales * kBytes);
    if constexpr (kForm == kIntZeros) __builtin_memcpy(&it.zero, r.zero + at, kScales);
  }

  // Scale (or zero point) s of a chunk.
  __device__ __forceinline__ static uint32_t field(const uint32_t* v, int s, int bytes) {
    const uint32_t x = v[s * bytes / 4];
    return bytes == 4 ? x : bytes == 2 ? (x >> 16 * (s & 1)) & 0xffffu : (x >> 8 * (s & 3)) & 0xffu;
  }

  // The last chunk of a K that is no multiple of 128, moved into place: codes behind the
  // row's last meet parts that are zero, and scales behind its last are zeros themselves
  // (another's could be infinite, which times a sum of zero is NaN).
  __device__ __forceinline__ void settle(It& it, int64_t k0) const {
    const int64_t want = k0 / 2 + 16 * (lane >> 4);
    // bytes, 16 and more: all behind
    const int by = (int)(want - min(want, (int64_t)row_bytes - 16));
    u32x4 v = it.codes;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if (by >> 2 > d)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < 3 ? v[i + 1] : 0u;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      it.codes[i] = __builtin_amdgcn_alignbyte(i < 3 ? v[i + 1] : 0u, v[i], by & 3);
    if constexpr (kScales > 1) {
      const int64_t at = k0 >> p.group_shift;
      const int shift = (int)(at - min(at, (int64_t)along - kScales));
      uint32_t s[kScales];
#pragma unroll
      for (int i = 0; i < kScales; ++i) {
        s[i] = 0;   // +0 as fp32, fp16 and bf16, 2^-127 as e8m0
#pragma unroll
        for (int j = 0; j < kScales; ++j)
          if (i + shift == j) s[i] = field(it.scale, j, kBytes);
      }
      uint32_t z = 0;
#pragma unroll
      for (int i = 0; i < (kScales * kBytes + 3) / 4; ++i) it.scale[i] = 0;
#pragma unroll
      for (int i = 0; i < kScales; ++i) {
        it.scale[i * kBytes / 4] |= s[i] << 8 * (i * kBytes % 4);
        if constexpr (kForm == kIntZeros)
          z |= ((it.zero >> 8 * min(i + shift, kScales - 1)) & 0xffu) << 8 * i;
      }
      if constexpr (kForm == kIntZeros) it.zero = z;
    }
  }

  // acc += this wave's chunk, whose parts begin at step step0 of those in LDS.
  __device__ __forceinline__ void multiply(It it, int chunk, int step0, float (&acc)[RT]) const {
    const int64_t k0 = (int64_t)chunk * kChunkK;
    if (__builtin_expect(k0 + kChunkK > K, 0)) settle(it, k0);
    const u32x4 codes = by_steps(it.codes);
    f32x4 sum[RT];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      constexpr int kPer = 4 / kScales;   // steps of a scale
      const int s = i / kPer;
      const float zero = kForm == kIntZeros ? (float)field(&it.zero, s, 1) : 8.f;
      const bf16x8 b = weights8<kForm, false>(codes[i], zero, 1.f);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const bf16x8 a = *reinterpret_cast<const bf16x8*>(own[t] + (step0 + i) * 64 * R);
        const f32x4 none = {0.f, 0.f, 0.f, 0.f};
        sum[t] = mfma16(a, b, i % kPer ? sum[t] : none);
      }
      if (i % kPer == kPer - 1) {
        const float scale = scale_value(field(it.scale, s, kBytes), kType);
        // a row's three parts first: one that is zero would be NaN by an infinite scale
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[t] += (sum[t][0] + (sum[t][1] + sum[t][2])) * scale;
      }
    }
  }

  // The parts of the chunks base .. base + here - 1: octet o, row q at (o R + q) 16.
  __device__ __forceinline__ void stage(int base, int here) const {
    const unsigned inverse = (65536 + rows - 1) / rows;   // u / rows for u below 65536 / 16
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
      u32x4 split[3];
      split8(x, split);
#pragma unroll
      for (int part = 0; part < 3; ++part)
        *reinterpret_cast<u32x4*>(parts + (octet * R + 3 * r + part) * 16) = split[part];
    }
  }

  __device__ __forceinline__ void put(const Epilogue& ep, int row, int64_t n, float v) const {
    const int to = row_to[row];
    if (n >= p.g.N || to < 0) return;
    float* out = p.g.C + to * p.g.ldc + n;
    *out = epilogue_apply(ep, row_of[row] >= 0 ? v : 0.f, out, n);
  }

  // The sums of a strip stored, those of the waves along K added: a lane has that of row
  // lane / 16 of each instruction.  Buffer 0 and 1 in turn.
  __device__ __forceinline__ void store(const Epilogue& ep, int strip, int buffer,
                                        const float (&v)[RT]) const {
    const int kw = 1 << kw_log2, wide = 16 * kWaves >> kw_log2;   // columns of the strip
    const int64_t n0 = (int64_t)strip * wide;
    if (kw == 1) {
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const int row = kRowsT * t + (lane >> 4);
        if (row < rows) put(ep, row, n0 + 16 * wave + (lane & 15), v[t]);
      }
      return;
    }
    // row r of wave w at (r / 4 * kWaves + w) 64 + r % 4 * 16
    float* red = reinterpret_cast<float*>(lds) + (buffers(RT) == 2 ? buffer * RT * kThreads : 0);
#pragma unroll
    for (int t = 0; t < RT; ++t) red[t * kThreads + tid] = v[t];
    __syncthreads();
    const int c = tid % wide;
    for (int r = tid / wide; r < rows; r += kThreads / wide) {
      const float* from = red + (r / kRowsT * kWaves + (c >> 4 << kw_log2)) * 64 +
                          r % kRowsT * 16 + (c & 15);
      float sum = 0.f;
#pragma unroll 8
      for (int i = 0; i < kw; ++i) sum += from[i * 64];
      put(ep, r, n0 + c, sum);
    }
    if (buffers(RT) == 1) __syncthreads();
  }

  // Places first .. first + rows - 1, every step-th strip from `strip` on.
  __device__ __forceinline__ void run(const Epilogue& ep, int first, int rows_, int strip,
                                      int step, int strips) {
    rows = rows_;
    R = 3 * rows;
    // (the fourth of a row, and rows behind the last, read another part: their sums are
    // not used)
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int q = 3 * (kRowsT * t + (lane >> 2 & 3)) + min(lane & 3, 2);
      own[t] = parts + ((lane >> 4) * R + min(q, R - 1)) * 16;
    }
    __syncthreads();   // the tile before is done with LDS
    if (tid < rows) {
      const int place = first + tid;
      const int r = p.g.ia ? p.g.ia[place] : place;
      row_of[tid] = r >= 0 && r < p.g.rows_a ? r : -1;
      const int to = p.g.ic ? p.g.ic[place] : place;
      row_to[tid] = to >= 0 && to < p.g.rows_c ? to : -1;
    }
    const int kw = 1 << kw_log2;
    pass = min(chunks, (kLdsBytes - sum_bytes(RT)) / (R * 256) & -kw);
    const int passes = (chunks + pass - 1) / pass;
    // positions: (strip, first chunk of the pass, this wave's place in it)
    struct Position {
      int strip, base, at;
    };
    auto advance = [&](Position& x) {
      x.at += kw;
      if ((x.at >> kw_log2) % kAhead == 0 && x.at >= min(pass, chunks - x.base)) {
        x.at = 0;
        x.base += pass;
        if (x.base >= chunks) {
          x.base = 0;
          x.strip += step;
        }
      }
    };
    It items[kAhead];
    Position now{strip, 0, 0}, ahead = now;
    Row row_ahead = row(strip);
    auto fetch_next = [&](It& it) {
      fetch(it, row_ahead, ahead.base + ahead.at + kwave);
      const int was = ahead.strip;
      advance(ahead);
      if (ahead.strip != was) row_ahead = row(ahead.strip);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      fetch_next(items[i]);
      // (out of order here, the first would be waited for behind the others in the loop)
      __builtin_amdgcn_sched_barrier(0);
    }
    float acc[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = 0.f;
    bool staged = false;
    int buffer = 0;
    // kAhead steps in turn, those behind a pass's chunks empty, so that staging and
    // storing, and the way out, stand here once: the code is fetched anew by each CU (by
    // the step they stand in it cost up to 1 us of 17; so do four steps).
    do {
      if (now.at == 0 && !staged) {
        __syncthreads();   // row_of is there; the pass before is used
        stage(now.base, min(pass, chunks - now.base));
        __syncthreads();
        staged = passes == 1;
      }
      const int was = now.strip;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int chunk = now.base + now.at + kwave;
        if (now.at + kwave < min(pass, chunks - now.base))
          multiply(items[i], chunk, (now.at + kwave) * 4, acc);
        fetch_next(items[i]);
        advance(now);
      }
      if (now.strip != was) {
        store(ep, was, buffer, acc);
        buffer ^= 1;
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[t] = 0.f;
      }
    } while (now.strip < strips);
  }
};

// Inclusive sum over the lanes of a wave, held at the largest value.
__device__ __forceinline__ unsigned scan_lanes(unsigned x) {
  const auto add = [&](auto ctrl, auto rows) {
    x = __builtin_elementwise_add_sat(
        x, (unsigned)__builtin_amdgcn_update_dpp(0, (int)x, ctrl.value, rows.value, 0xf, false));
  };
  // 1, 2, 4 and 8 lanes up in rows of 16; row 0 (2) into row 1 (3), both into the others
  add(std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xf>{});
  add(std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xf>{});
  add(std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xf>{});
  add(std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xf>{});
  add(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xa>{});
  add(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xc>{});
  return x;
}

// The row tiles of all groups in order.  A lane has a group, each wave the same ones and
// nothing to wait for, up to 64 of them; with more a thread has a group, so that any number
// takes one load and one sum over the workgroup (0.5 us more).
struct GroupTiles {
  unsigned first, tiles;   // of this lane's or thread's group
  int begin, rows;
  unsigned total;          // of all
  bool waves;              // each alone
  struct Shared {
    unsigned sums[kWaves];
    int found[3];
  };
  static_assert(kMaxGroups <= kThreads, "a thread for each group");

  __device__ __forceinline__ void find_all(const Q4Problem& p, Shared& lds) {
    waves = p.g.groups <= 64;
    const int wave = threadIdx.x >> 6, g = waves ? threadIdx.x & 63 : threadIdx.x;
    begin = rows = 0;
    if (g < p.g.groups) {
      int end;
      group_span(p.g.offsets, g, p.g.rows, begin, end);
      rows = end - begin;
    }
    tiles = q4_few_rows(p) == kQ4FewRows
                ? ((unsigned)rows + kQ4FewRows - 1) / kQ4FewRows
                : ((unsigned)rows + kQ4FewRowsDeep - 1) / kQ4FewRowsDeep;
    const unsigned incl = scan_lanes(tiles);
    first = incl - tiles;
    total = __builtin_amdgcn_readlane(incl, 63);
    if (waves) return;
    if ((g & 63) == 63) lds.sums[wave] = incl;
    __syncthreads();
    unsigned before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w == wave) before = total;
      total = __builtin_elementwise_add_sat(total, lds.sums[w]);
    }
    first = __builtin_elementwise_add_sat(first, before);
    total = __builtin_amdgcn_readfirstlane(total);
  }

  // Row tile t's group, its first place and rows: a group's tiles have one size.
  __device__ __forceinline__ void find(unsigned t, Shared& lds, int& group, int& place,
                                       int& count) const {
    const bool here = t >= first && t - first < tiles;
    const int each = tiles <= 1 ? rows : (int)(((unsigned)rows + tiles - 1) / tiles);
    const int at = here ? (int)(t - first) * each : 0;
    place = begin + at;
    count = min(each, rows - at);
    if (waves) {
      const int lane = __builtin_ctzll(__builtin_amdgcn_ballot_w64(here));
      group = lane;
      place = __builtin_amdgcn_readlane(place, lane);
      count = __builtin_amdgcn_readlane(count, lane);
      return;
    }
    if (here) {
      lds.found[0] = threadIdx.x;
      lds.found[1] = place;
      lds.found[2] = count;
    }
    __syncthreads();
    group = __builtin_amdgcn_readfirstlane(lds.found[0]);
    place = __builtin_amdgcn_readfirstlane(lds.found[1]);
    count = __builtin_amdgcn_readfirstlane(lds.found[2]);
  }
};

// Quotient of numbers up to 256, rounded down: a + 1/2 over b is at least 2^-9 from the whole
// numbers, the reciprocal and the product are off by 2^-14 at most.
__device__ __forceinline__ unsigned small_quotient(unsigned a, unsigned b) {
  return (unsigned)(((float)a + 0.5f) * __builtin_amdgcn_rcpf((float)b));
}

// A row tile goes to as many workgroups as there are CUs for it, which take its strips in
// turn; further tiles follow after one another.  Without offsets the host says how many
// (tiles along the grid's y, of `each` rows).  With them only the device can: 192 rows of 32
// groups of 2048 x 1024 are 32 tiles, which take 18 us, or, all in one group, 10, which take
// 23 (183 with each group's tiles one after another on workgroups of its own).
template <int kForm, int kScales, int kType>
__global__ void __launch_bounds__(kThreads, 4)
    q4_few_kernel(Q4Problem p, Epilogue ep, unsigned tiles, int each) {
  __shared__ __attribute__((aligned(16))) char lds[kLdsBytes];
  __shared__ int row_of[2 * kQ4FewRows];
  __shared__ GroupTiles::Shared shared;
  const int strips = q4_few_strips(p);
  unsigned tile = blockIdx.y, share = blockIdx.x, per = gridDim.x, step = gridDim.y;
  GroupTiles all;
  if (p.g.offsets) {
    all.find_all(p, shared);
    tiles = all.total;
    if (tiles == 0) return;
    per = min(tiles < kQ4Cus ? small_quotient(kQ4Cus, tiles) : 1u, (unsigned)strips);
    tile = small_quotient(blockIdx.x, per);
    share = blockIdx.x - tile * per;
    step = kQ4Cus;
  }
  for (; tile < tiles; tile += step) {
    int group = 0, place = (int)tile * each, rows = min(each, p.g.rows - place);
    if (p.g.offsets) all.find(tile, shared, group, place, rows);
    Epilogue e = ep;
    if (e.bias) e.bias += group * p.g.sbias;
    auto run = [&](auto few) { few.run(e, place, rows, (int)share, (int)per, strips); };
    if (rows <= kRowsT)
      run(Few<1, kForm, kScales, kType>(p, group, lds, row_of));
    else if (rows <= 2 * kRowsT)
      run(Few<2, kForm, kScales, kType>(p, group, lds, row_of));
    else if (rows <= 3 * kRowsT)
      run(Few<3, kForm, kScales, kType>(p, group, lds, row_of));
    else if (rows <= 4 * kRowsT)
      run(Few<4, kForm, kScales, kType>(p, group, lds, row_of));
    else
      run(Few<5, kForm, kScales, kType>(p, group, lds, row_of));
  }
}

template <int kForm, int kScales, int kType>
hipError_t launch(const Q4Problem& p, const Epilogue& e, hipStream_t s) {
  const int most = q4_few_rows(p);
  dim3 grid(kQ4Cus);   // a workgroup a CU
  unsigned tiles = 0, each = 0;
  if (!p.g.offsets) {
    tiles = ((unsigned)p.g.rows + most - 1) / most;
    each = ((unsigned)p.g.rows + tiles - 1) / tiles;
    grid = dim3(std::min(std::max(1u, kQ4Cus / tiles), (unsigned)q4_few_strips(p)),
                std::min(tiles, 1024u));
  }
  q4_few_kernel<kForm, kScales, kType><<<grid, kThreads, 0, s>>>(p, e, tiles, (int)each);
  return hipGetLastError();
}

template <int kForm, int kScales>
hipError_t by_type(const Q4Problem& p, const Epilogue& e, hipStream_t s) {
  if (p.scale_type == kScaleF32) return launch<kForm, kScales, kScaleF32>(p, e, s);
  if (p.scale_type == kScaleE8m0) return launch<kForm, kScales, kScaleE8m0>(p, e, s);
  if (p.scale_type == kScaleBf16) return launch<kForm, kScales, kScaleBf16>(p, e, s);
  return launch<kForm, kScales, kScaleF16>(p, e, s);
}
template <int kForm>
hipError_t by_group(const Q4Problem& p, const Epilogue& e, hipStream_t s) {
  if (p.group_shift == 5) return by_type<kForm, 4>(p, e, s);
  if (p.group_shift == 6) return by_type<kForm, 2>(p, e, s);
  return by_type<kForm, 1>(p, e, s);
}

}  // namespace

hipError_t launch_q4_few(const Q4Problem& p, const Epilogue& e, hipStream_t s) {
  if (p.g.K < kChunkK) return hipErrorInvalidValue;
  return p.e2m1 ? by_group<kE2m1>(p, e, s)
                : p.zero ? by_group<kIntZeros>(p, e, s) : by_group<kInt8>(p, e, s);
}

}  // namespace gemmf32
