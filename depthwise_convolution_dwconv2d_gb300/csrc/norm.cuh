// Device helpers shared by the group-norm kernels: vectors of channels from
// any source, the normalised value, activations and their slopes.
#pragma once

#include "dependent.cuh"
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

// 2^v and 1 / v by the special-function unit: 2 and 1 units in the last place, results below 2^-126 flushed to 0
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ f32x2 both(float v) { return pack_f32x2(v, v); }
__device__ __forceinline__ f32x2 neg(f32x2 v) { return v ^ 0x8000000080000000ull; }
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  fma_f32x2(c, a, b);
  return c;
}

// 1 / (1 + exp(-c v)) of both lanes; c2 = -c log2(e). The product is rounded
// before the power is taken, so far out on the negative side the result is
// off by about |c v| * 2^-24 of itself.
__device__ __forceinline__ f32x2 sigmoid2(f32x2 v, float c2) {
  float a, b;
  unpack_f32x2(mul_f32x2(v, both(c2)), a, b);
  unpack_f32x2(add_f32x2(pack_f32x2(exp2_fast(a), exp2_fast(b)), both(1.f)), a, b);
  return pack_f32x2(rcp_fast(a), rcp_fast(b));
}
constexpr float kLog2e = 1.4426950408889634f;

// act(u) and act'(u) of both lanes; NaN stays NaN
template <int ACT>
__device__ __forceinline__ f32x2 act_of(f32x2 u) {
  if (ACT == DWCONV_ACT_SILU) return mul_f32x2(u, sigmoid2(u, -kLog2e));
  if (ACT == DWCONV_ACT_GELU) {
    const f32x2 w = mul_f32x2(u, fma2(mul_f32x2(u, u), both(kCubic), both(1.f)));  // u + 0.044715 u^3
    return mul_f32x2(u, sigmoid2(w, -kGelu * kLog2e));
  }
  float a, b;
  unpack_f32x2(u, a, b);
  if (ACT == DWCONV_ACT_RELU || ACT == DWCONV_ACT_RELU6) {
    a = a < 0.f ? 0.f : a;
    b = b < 0.f ? 0.f : b;
  }
  if (ACT == DWCONV_ACT_RELU6) {
    a = a > 6.f ? 6.f : a;
    b = b > 6.f ? 6.f : b;
  }
  return pack_f32x2(a, b);
}
template <int ACT>
__device__ __forceinline__ f32x2 slope_of(f32x2 u) {
  if (ACT == DWCONV_ACT_SILU) {  // q (1 + u (1 - q))
    const f32x2 q = sigmoid2(u, -kLog2e);
    return mul_f32x2(q, fma2(u, add_f32x2(both(1.f), neg(q)), both(1.f)));
  }
  if (ACT == DWCONV_ACT_GELU) {  // q (1 + u (1 - q) 2 sqrt(2 / pi) (1 + 3 * 0.044715 u^2))
    const f32x2 uu = mul_f32x2(u, u);
    const f32x2 q = sigmoid2(mul_f32x2(u, fma2(uu, both(kCubic), both(1.f))), -kGelu * kLog2e);
    const f32x2 w = mul_f32x2(u, fma2(uu, both(3.f * kGelu * kCubic), both(kGelu)));
    return mul_f32x2(q, fma2(w, add_f32x2(both(1.f), neg(q)), both(1.f)));
  }
  float a, b;
  unpack_f32x2(u, a, b);
  if (ACT == DWCONV_ACT_RELU) return pack_f32x2(a > 0.f ? 1.f : 0.f, b > 0.f ? 1.f : 0.f);
  if (ACT == DWCONV_ACT_RELU6)
    return pack_f32x2(a > 0.f && a < 6.f ? 1.f : 0.f, b > 0.f && b < 6.f ? 1.f : 0.f);
  return both(1.f);
}

// NP pairs at a time: one uniform branch per vector
template <int NP>
__device__ __forceinline__ void act_p(int act, f32x2* u) {
#define X(A)                                                  \
  case A:                                                     \
    _Pragma("unroll") for (int e = 0; e < NP; ++e) u[e] = act_of<A>(u[e]); \
    break;
  switch (act) { X(DWCONV_ACT_RELU) X(DWCONV_ACT_RELU6) X(DWCONV_ACT_SILU) X(DWCONV_ACT_GELU) default: break; }
#undef X
}
// u <- act'(u)
template <int NP>
__device__ __forceinline__ void slope_p(int act, f32x2* u) {
#define X(A)                                                  \
  case A:                                                     \
    _Pragma("unroll") for (int e = 0; e < NP; ++e) u[e] = slope_of<A>(u[e]); \
    break;
  switch (act) { X(DWCONV_ACT_RELU) X(DWCONV_ACT_RELU6) X(DWCONV_ACT_SILU) X(DWCONV_ACT_GELU) default: X(DWCONV_ACT_NONE) }
#undef X
}

// the same of V values held one by one
template <int V>
__device__ __forceinline__ void act_v(int act, float* u) {
  f32x2 p[(V + 1) / 2];
#pragma unroll
  for (int e = 0; e < (V + 1) / 2; ++e) p[e] = pack_f32x2(u[2 * e], 2 * e + 1 < V ? u[2 * e + 1] : 0.f);
  act_p<(V + 1) / 2>(act, p);
#pragma unroll
  for (int e = 0; e < (V + 1) / 2; ++e) {
    float a, b;
    unpack_f32x2(p[e], a, b);
    u[2 * e] = a;
    if (2 * e + 1 < V) u[2 * e + 1] = b;
  }
}
template <int V>
__device__ __forceinline__ void slope_v(int act, float* u) {
  f32x2 p[(V + 1) / 2];
#pragma unroll
  for (int e = 0; e < (V + 1) / 2; ++e) p[e] = pack_f32x2(u[2 * e], 2 * e + 1 < V ? u[2 * e + 1] : 0.f);
  slope_p<(V + 1) / 2>(act, p);
#pragma unroll
  for (int e = 0; e < (V + 1) / 2; ++e) {
    float a, b;
    unpack_f32x2(p[e], a, b);
    u[2 * e] = a;
    if (2 * e + 1 < V) u[2 * e + 1] = b;
  }
}

}  // namespace norm
}  // namespace dwconv
