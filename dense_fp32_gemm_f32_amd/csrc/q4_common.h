// What the kernels of the products with 4-bit weights share.
//
// An fp32 value is the sum of three bf16 values exactly (its 24 significant bits
// in three times 8), and a 4-bit weight without its scale, code - zero or the e2m1
// value, is one bf16 value exactly.  So the fp32 product is three bf16 products
// whose terms are exact and whose sums the matrix instruction holds in fp32, at a
// third of the bf16 rate (about 450 TFLOP/s by the library's own 1350) where the
// fp32 matrix instruction has 157.  The scale is the group's: a group's sum is
// formed without it and added, times the scale, to the output's sum in fp32.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "experts_internal.h"

namespace gemmf32 {
namespace q4 {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// The high halves of b and a, a's below b's.
__device__ __forceinline__ uint32_t high_halves(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

// Eight fp32 values as three times eight bf16 values (parts[0] the highest), each
// rounded to nearest from what the parts before it leave: the remainders, formed two
// at a time by the bf16 dot product that adds to an fp32 value, are exact (a part
// below the smallest normal float counts as zero).  In octets with a value that is
// not finite, or rounds to infinity, the parts are cut off instead of rounded, and a
// value that is not finite has itself as its first part and zeros behind it.
__device__ __forceinline__ void split8(const float (&x)[8], u32x4 (&parts)[3]) {
  // (-1, 0) and (0, -1), in registers: as an inline constant the instruction takes
  // -1 for the fp32 bits
  uint32_t c0 = 0x0000bf80u, c1 = 0xbf800000u;
  asm("" : "+v"(c0), "+v"(c1));
  const bf16x2 low = __builtin_bit_cast(bf16x2, c0), high = __builtin_bit_cast(bf16x2, c1);
  const bf16x2 none = {(__bf16)0.f, (__bf16)0.f};
  float y[8], probe = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = x[i];
#pragma unroll
  for (int part = 0; part < 3; ++part) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 two = {y[2 * i], y[2 * i + 1]};
      const bf16x2 h = __builtin_convertvector(two, bf16x2);
      parts[part][i] = __builtin_bit_cast(uint32_t, h);
      if (part < 2) {
        y[2 * i] = __builtin_amdgcn_fdot2_f32_bf16(h, low, y[2 * i], false);
        y[2 * i + 1] = __builtin_amdgcn_fdot2_f32_bf16(h, high, y[2 * i + 1], false);
      } else {
        probe = __builtin_amdgcn_fdot2_f32_bf16(h, none, probe, false);   // NaN there: NaN
      }
    }
  }
  if (__builtin_expect(__ballot(probe != 0.f) != 0, 0)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = x[i];
      asm volatile("" : "+v"(v));   // keeps all of this in the branch
      const uint32_t u = __float_as_uint(v);
      const bool finite = (u & 0x7f800000u) != 0x7f800000u;
      // a NaN stays one with its low bits cut off
      uint32_t h = (u & 0xffff0000u) | (!finite && (u & 0x7fffffu) ? 0x400000u : 0u);
#pragma unroll
      for (int part = 0; part < 3; ++part) {
        const uint32_t keep = i & 1 ? 0x0000ffffu : 0xffff0000u;
        parts[part][i / 2] = (parts[part][i / 2] & keep) | (i & 1 ? h & 0xffff0000u : h >> 16);
        v = finite ? v - __uint_as_float(h) : 0.f;
        h = __float_as_uint(v) & 0xffff0000u;
      }
    }
  }
}

// What codes stand for: int with the zero point 8, int with zero points, e2m1.
enum Form { kInt8, kIntZeros, kE2m1 };

// Eight weights from a dword of codes (the first k in its low bits), without their
// scale, or with a scale that is a power of two (kScaled): bf16 values exactly.  int
// codes: read as e4m3 with a scale of 2^9, the bytes 0 .. 15 are the values 0 .. 15
// (the format is linear there), so that one instruction converts two; minus the
// zero point they are whole numbers of at most 8 bits.
template <int kForm, bool kScaled>
__device__ __forceinline__ bf16x8 weights8(uint32_t x, float zero, float scale) {
  u32x4 w;
  const float by = kScaled ? scale : 1.f;
  if constexpr (kForm == kE2m1) {
    bf16x2 v[4];
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, by, 0);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, by, 1);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, by, 2);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, by, 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __builtin_bit_cast(uint32_t, v[i]);
  } else {
    const uint32_t lo = x & 0x0f0f0f0fu, hi = (x >> 4) & 0x0f0f0f0fu;
    const f32x2 e0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, 512.f, false),
                e1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, 512.f, true),
                o0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, 512.f, false),
                o1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, 512.f, true);
    auto value = [&](float c) { return kScaled ? (c - zero) * by : c - zero; };
    w[0] = high_halves(value(e0[0]), value(o0[0]));
    w[1] = high_halves(value(e0[1]), value(o0[1]));
    w[2] = high_halves(value(e1[0]), value(o1[0]));
    w[3] = high_halves(value(e1[1]), value(o1[1]));
  }
  return __builtin_bit_cast(bf16x8, w);
}

// Entry i of the scales as it is stored, and its value.  (Loads that are to stay in
// flight must not be looked at: a conversion beside the load would wait for all.)
__device__ __forceinline__ uint32_t load_scale(const void* scale, int type, int64_t i) {
  if (type == kScaleF32) return static_cast<const uint32_t*>(scale)[i];
  if (type == kScaleE8m0) return static_cast<const uint8_t*>(scale)[i];
  return static_cast<const uint16_t*>(scale)[i];
}
__device__ __forceinline__ float scale_value(uint32_t bits, int type) {
  if (type == kScaleF32) return __uint_as_float(bits);
  if (type == kScaleF16) return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  if (type == kScaleBf16) return __uint_as_float(bits << 16);
  // e8m0, the exponent of a power of two; 255 is NaN
  return __uint_as_float(bits == 255 ? 0x7fc00000u : bits == 0 ? 0x00400000u : bits << 23);
}

// Lane group g (16 lanes) has dwords 0 .. 3 of codes 32 g + 0 .. 31; afterwards
// dword i holds codes 32 i + 8 g + 0 .. 7: the transposition of four groups and
// four registers.
__device__ __forceinline__ u32x4 by_steps(u32x4 v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// One group's matrix of weights.
struct Weights {
  const uint8_t* codes;
  const uint8_t* zero;   // NULL: 8
  const void* scale;
  int64_t scale0;        // entry of row 0, group 0
  __device__ __forceinline__ Weights(const Q4Problem& p, int g)
      : codes(p.codes + g * p.sq),
        zero(p.zero ? p.zero + g * p.sz : nullptr),
        scale(p.scale),
        scale0(g * p.ss) {}
};

}  // namespace q4
}  // namespace gemmf32
