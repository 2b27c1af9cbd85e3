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


// The weight of a key times its value's scale, p vs, is rounded to fp16, so a row's reference n (p = 2^(z - n)) has
// to follow the largest z + log2 vs over its keys: jointly, since a key with a large logit and a small value
// (attention sinks are such keys) would push the others below fp16's least number, where each loses what the sum l
// counts.  WEIGHT_ROOM: the reference stays so far (log2) below that maximum, and is raised when the maximum has
// grown by 2^8 past it.  Products thus reach 2^15 of fp16's 2^16, and half of its least number is at most 2^-32 of
// the row's largest product, where without the room it is 2^-25: over 2^17 keys that adds up to 2^-8.
// SCALE_FLOOR: what log2 vs counts as for values of 0 and of less.  p is then at most 2^(8 + 7 + 87), and its sum over
// a prefix (fewer than 2^25 keys) below 2^127.
constexpr float WEIGHT_ROOM = 7.f, SCALE_FLOOR = -87.f;

// What a key's value scale adds to its logit (log2) for the reference.  A scale that is no number says nothing about
// the weights (an infinite reference would make all of them 0): it shows in the products.
__device__ __forceinline__ float scale_log2(float vs) {
  const float x = fast_log2(fabsf(vs));
  return (x < 128.f ? fmaxf(x, SCALE_FLOOR) : SCALE_FLOOR) - WEIGHT_ROOM;
}

}  // namespace pisa
