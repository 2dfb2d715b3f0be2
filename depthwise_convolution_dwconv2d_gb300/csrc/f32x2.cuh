// Products and sums of two-lane fp32 operands (f32x2, common.cuh).
#pragma once

#include "common.cuh"

namespace dwconv {

// d = a * b and a + b on both lanes, each lane rounded by itself
__device__ __forceinline__ f32x2 mul_f32x2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 add_f32x2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// a + b lane by lane, for an addend that is a packed product: the assembler
// contracts mul.rn.f32x2 and add.rn.f32x2 into one rounding (seen in codes
// next to a tie), which the scalar addition prevents.
__device__ __forceinline__ f32x2 add_apart(f32x2 a, f32x2 b) {
  float a0, a1, b0, b1;
  unpack_f32x2(a, a0, a1);
  unpack_f32x2(b, b0, b1);
  return pack_f32x2(__fadd_rn(a0, b0), __fadd_rn(a1, b1));
}

}  // namespace dwconv
