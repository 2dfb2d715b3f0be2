// Device helpers shared by the group-norm kernels: vectors of channels from
// any source, the normalised value, activations and their slopes.
#pragma once

#include "norm.h"
#include "vec.cuh"

namespace dwconv {
namespace norm {

// V channels (16 bytes, or one element) of the storage type <-> fp32
template <typename T, int V>
__device__ __forceinline__ void load_v(const T* p, float* o) {
  if constexpr (V == 1) {
    o[0] = to_f<T>(*p);
  } else {
    unpack16<T>(*reinterpret_cast<const uint4*>(p), o);
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float* f) {
  if constexpr (V == 1) {
    *p = from_f<T>(f[0]);
  } else {
    *reinterpret_cast<uint4*>(p) = pack16<T>(f);
  }
}

// V values of a checkpoint at (row, channel c); V divides the block
template <int SRC, int V>
__device__ __forceinline__ void load_act8(const Act8& t, int64_t row, int C, int c, float* o) {
  const uint8_t* p = t.codes + row * C + c;
  const float s = __ldg(t.scales + row * t.nblk + (c >> t.shift));
  if constexpr (V == 1) {
    o[0] = code1<SRC>(*p);
  } else if constexpr (V == 4) {
    codes4<SRC>(*reinterpret_cast<const uint32_t*>(p), o);
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    codes4<SRC>(u.x, o);
    codes4<SRC>(u.y, o + 4);
  }
#pragma unroll
  for (int e = 0; e < V; ++e) o[e] = __fmul_rn(o[e], s);
}

// xh and u with each operation rounded by itself: forward and backward then
// agree, bit for bit, on which side of a kink of the activation u lies.
__device__ __forceinline__ float xhat(float x, float mean, float rstd) {
  return __fmul_rn(__fsub_rn(x, mean), rstd);
}
__device__ __forceinline__ float affine(float xh, float gamma, float beta) {
  return __fadd_rn(__fmul_rn(xh, gamma), beta);
}

constexpr float kGelu = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kCubic = 0.044715f;

// 1 / (1 + exp(-v)) with the fast exponential and division: a few units in
// the last place, and 0 where exp(-v) overflows
__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// act(u); NaN stays NaN
template <int ACT>
__device__ __forceinline__ float act_of(float u) {
  if (ACT == DWCONV_ACT_RELU) return u < 0.f ? 0.f : u;
  if (ACT == DWCONV_ACT_RELU6) return u < 0.f ? 0.f : (u > 6.f ? 6.f : u);
  if (ACT == DWCONV_ACT_SILU) return __fdividef(u, 1.f + __expf(-u));
  if (ACT == DWCONV_ACT_GELU) return __fdividef(u, 1.f + __expf(-kGelu * (u + kCubic * u * u * u)));
  return u;
}

// act'(u)
template <int ACT>
__device__ __forceinline__ float slope_of(float u) {
  if (ACT == DWCONV_ACT_RELU) return u > 0.f ? 1.f : 0.f;
  if (ACT == DWCONV_ACT_RELU6) return u > 0.f && u < 6.f ? 1.f : 0.f;
  if (ACT == DWCONV_ACT_SILU) {
    const float q = sigmoid(u);
    return q * (1.f + u * (1.f - q));
  }
  if (ACT == DWCONV_ACT_GELU) {
    const float q = sigmoid(kGelu * (u + kCubic * u * u * u));
    return q + u * q * (1.f - q) * (kGelu * (1.f + 3.f * kCubic * u * u));
  }
  return 1.f;
}

// V values at a time: one uniform branch per vector
template <int V>
__device__ __forceinline__ void act_v(int act, float* u) {
#define X(A)                                                  \
  case A:                                                     \
    _Pragma("unroll") for (int e = 0; e < V; ++e) u[e] = act_of<A>(u[e]); \
    break;
  switch (act) { X(DWCONV_ACT_RELU) X(DWCONV_ACT_RELU6) X(DWCONV_ACT_SILU) X(DWCONV_ACT_GELU) default: break; }
#undef X
}

// u <- act'(u)
template <int V>
__device__ __forceinline__ void slope_v(int act, float* u) {
#define X(A)                                                  \
  case A:                                                     \
    _Pragma("unroll") for (int e = 0; e < V; ++e) u[e] = slope_of<A>(u[e]); \
    break;
  switch (act) { X(DWCONV_ACT_NONE) X(DWCONV_ACT_RELU) X(DWCONV_ACT_RELU6) X(DWCONV_ACT_SILU) X(DWCONV_ACT_GELU) default: break; }
#undef X
}

}  // namespace norm
}  // namespace dwconv
