// 8-bit activation checkpoints: one code per value and one fp32 scale per
// block of 32, 64 or 128 channels of a row. Code arithmetic shared by the
// kernels that write and read them.
//
//   scale = fl(max|x| * fl(1 / Q)),  code = nearest(fl(x * fl(1 / scale))),
//   value = fl(code * scale),        Q = 127 (integers) or 448 (e4m3)
//
// max|x| is taken on the bit patterns without the sign, as integers: it needs
// no rounding, so its order is free, and it keeps infinities and NaN (both
// above every finite pattern). From an infinite or NaN maximum the scale is
// infinite or NaN, every code is 0 or NaN, and 0 * inf = NaN: the block
// decodes to NaN.
#pragma once

#include "common.cuh"

namespace dwconv {

// What holds the input of a kernel: the storage type, or codes.
enum Src : int { kSrcFull = 0, kSrcI8 = 1, kSrcE4M3 = 2 };

// A checkpoint, passed to kernels by value.
struct Act8 {
  uint8_t* codes;
  float* scales;
  int src;    // kSrcI8 or kSrcE4M3
  int shift;  // log2 of the block
  int nblk;   // scales per row
};

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// scale and its reciprocal from the block's largest pattern (0 / 0 for a
// block of zeros or of values too small for a normal scale)
template <int SRC>
__device__ __forceinline__ float scale_of(uint32_t amax_bits, float* inv) {
  constexpr float r = SRC == kSrcI8 ? 1.0f / 127.0f : 1.0f / 448.0f;
  const float s = __fmul_rn(__uint_as_float(amax_bits), r);
  const bool zero = s < 1.17549435e-38f;  // false for NaN
  *inv = zero ? 0.f : __frcp_rn(s);
  return zero ? 0.f : s;
}

// four values -> four codes, first value in the low byte
template <int SRC>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv) {
  a = __fmul_rn(a, inv);
  b = __fmul_rn(b, inv);
  c = __fmul_rn(c, inv);
  d = __fmul_rn(d, inv);
  if (SRC == kSrcI8) {
    // |v| is at most 127 (1 + 2^-22), so the nearest integer fits a byte; NaN converts to 0
    const uint32_t p = __byte_perm((uint32_t)__float2int_rn(a), (uint32_t)__float2int_rn(b), 0x0040);
    const uint32_t q = __byte_perm((uint32_t)__float2int_rn(c), (uint32_t)__float2int_rn(d), 0x0040);
    return __byte_perm(p, q, 0x5410);
  }
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

template <int SRC>
__device__ __forceinline__ uint8_t encode1(float a, float inv) {
  return (uint8_t)(encode4<SRC>(a, 0.f, 0.f, 0.f, inv) & 0xffu);
}

// two codes (low 16 bits) -> two unscaled values, exact
__device__ __forceinline__ void e4m3_pair(uint16_t v, float& a, float& b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  a = f.x;
  b = f.y;
}

// four codes -> four unscaled values, exact. An integer code c is read as
// the float 2^23 + (c + 128), from which 2^23 + 128 is subtracted: a byte
// move and an addition instead of a conversion.
template <int SRC>
__device__ __forceinline__ void codes4(uint32_t v, float* o) {
  if (SRC == kSrcI8) {
    const uint32_t u = v ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7650 + i)) - 8388736.0f;
  } else {
    e4m3_pair((uint16_t)(v & 0xffffu), o[0], o[1]);
    e4m3_pair((uint16_t)(v >> 16), o[2], o[3]);
  }
}

// one code -> its unscaled value, exact
template <int SRC>
__device__ __forceinline__ float code1(uint8_t c) {
  float o[4];
  codes4<SRC>((uint32_t)c, o);
  return o[0];
}

// act8.cu. x and the checkpoint share rows x C; x's rows are ldx values apart.
cudaError_t act8_encode(int64_t rows, int64_t C, int64_t ldx, int dtype, const void* x, const Act8& t,
                        cudaStream_t s);
cudaError_t act8_decode(int64_t rows, int64_t C, int64_t ldx, int dtype, const Act8& t, void* x,
                        cudaStream_t s);

}  // namespace dwconv
