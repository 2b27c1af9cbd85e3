// int8 codes as fp16 operands: what the kernels that attend over the 8-bit cache have in common.
#pragma once

#include "common.cuh"

namespace pisa {

// Two codes with their top bit flipped (code + 128) in two bytes of x -> fp16x2: 0x6400 | u is 1024 + u.
template <int SEL>
__device__ __forceinline__ uint32_t widen_f16(uint32_t x) {
  const uint32_t y = __byte_perm(x, 0x64646464u, SEL);
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(y), "r"(0x64806480u));  // 1152
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace pisa
