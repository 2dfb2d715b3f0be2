// 8-bit activation checkpoints: one code per value and one fp32 scale per
// block of 32, 64 or 128 channels of a row. Code arithmetic shared by the
// kernels that write and read them.
//
//   scale = fl(max|x| * fl(1 / Q)),  code = nearest(fl(x * fl(1 / scale))),
//   value = fl(code * scale),        Q = 127 (integers) or 448 (e4m3)
//
// max|x| is taken on the bit patterns without the sign, as integers: it needs
// no rounding, so its order is free, and it keeps infinities and NaN (both
// above every finite pattern): their block's scale is NaN, and so is every
// value decoded from it.
#pragma once

#include "f32x2.cuh"

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

// The largest pattern without sign of a vector's values and its neighbours'
// of a block of channels (`lanes` of them), as that of an fp32 value.
// Patterns of 16-bit types are compared two at a time.
template <typename T, int V, typename W>
__device__ __forceinline__ uint32_t block_max(W w, int lanes) {
  const uint32_t* u = reinterpret_cast<const uint32_t*>(&w);
  uint32_t m = 0;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < V; ++e) m = max(m, u[e] & 0x7fffffffu);
    for (int o = lanes >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
  } else {
#pragma unroll
    for (int e = 0; e < V / 2; ++e) m = __vmaxu2(m, u[e] & 0x7fff7fffu);
    for (int o = lanes >> 1; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    const unsigned short h = (unsigned short)max(m & 0xffffu, m >> 16);
    return __float_as_uint(to_f<T>(*reinterpret_cast<const T*>(&h)));
  }
}

// scale and its reciprocal from the block's largest pattern (0 / 0 for a
// block of zeros or of values too small for a normal scale)
template <int SRC>
__device__ __forceinline__ float scale_of(uint32_t amax_bits, float* inv) {
  constexpr float r = SRC == kSrcI8 ? 1.0f / 127.0f : 1.0f / 448.0f;
  const float s = __fmul_rn(__uint_as_float(amax_bits), r);
  const bool zero = s < 1.17549435e-38f;  // false for NaN
  *inv = zero ? 0.f : __frcp_rn(s);
  return zero ? 0.f : (amax_bits >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : s);
}

// four values (two pairs) -> four codes, first value in the low byte. The
// integer nearest to v (|v| is at most 127 (1 + 2^-22)) is the low byte of
// v + 1.5 * 2^23: an addition, which rounds to nearest even, instead of a
// conversion.
template <int SRC>
__device__ __forceinline__ uint32_t encode4(f32x2 ab, f32x2 cd, float inv) {
  const f32x2 i2 = pack_f32x2(inv, inv);
  ab = mul_f32x2(ab, i2);
  cd = mul_f32x2(cd, i2);
  float a, b, c, d;
  if (SRC == kSrcI8) {
    const f32x2 magic = pack_f32x2(12582912.f, 12582912.f);
    unpack_f32x2(add_apart(ab, magic), a, b);
    unpack_f32x2(add_apart(cd, magic), c, d);
    return __byte_perm(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040),
                       __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040), 0x5410);
  }
  unpack_f32x2(ab, a, b);
  unpack_f32x2(cd, c, d);
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
template <int SRC>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv) {
  return encode4<SRC>(pack_f32x2(a, b), pack_f32x2(c, d), inv);
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

// four codes -> four values (two pairs)
template <int SRC>
__device__ __forceinline__ void decode4(uint32_t v, float scale, f32x2* o) {
  const f32x2 s2 = pack_f32x2(scale, scale);
  if (SRC == kSrcI8) {
    const uint32_t u = v ^ 0x80808080u;
    const f32x2 bias = pack_f32x2(-8388736.0f, -8388736.0f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x2 m = pack_f32x2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7650 + 2 * i)),
                                 __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7651 + 2 * i)));
      o[i] = mul_f32x2(add_f32x2(m, bias), s2);
    }
  } else {
    float f[4];
    e4m3_pair((uint16_t)(v & 0xffffu), f[0], f[1]);
    e4m3_pair((uint16_t)(v >> 16), f[2], f[3]);
    o[0] = mul_f32x2(pack_f32x2(f[0], f[1]), s2);
    o[1] = mul_f32x2(pack_f32x2(f[2], f[3]), s2);
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
