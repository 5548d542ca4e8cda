// Direct global -> LDS copy for the gfx950 MFMA kernels.
#pragma once

#include <cstdint>

#include <hip/hip_runtime.h>

namespace gemmf32 {
namespace mfma {

// One global_load_lds_dwordx4: lane l copies 16 bytes from g into LDS at
// lds_wave + 16 l (lds_wave is the same for the whole wave).  The instruction
// takes its LDS address (the low half of the pointer) from M0, and needs one
// wait state behind a scalar write of M0.  The compiler puts the address there,
// but sees no load in the string whose wait it would keep: hence the s_nop.
// (With M0 saved, written and restored inside the string 4096^3 takes 954 us
// instead of 925.)
//
// It is written as inline assembly on purpose: the compiler cannot tell which
// LDS buffer a load through its builtin writes, and so makes every later LDS
// read wait for all loads still in flight, including loads into the other
// buffer.  The kernels wait themselves (s_waitcnt vmcnt(0) before the barrier
// that publishes a buffer), so reads of one buffer overlap loads into the
// other.
__device__ __forceinline__ void load_lds16(const float* g, float* lds_wave) {
  const uint32_t lds_addr = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds_wave);
  asm volatile(
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %0, off"
      :
      : "v"(g), "{m0}"(lds_addr)
      : "memory");
}

}  // namespace mfma
}  // namespace gemmf32
