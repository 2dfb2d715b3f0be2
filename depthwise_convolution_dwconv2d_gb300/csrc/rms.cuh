// Helpers shared by the RMS norm's forward and backward kernels.
#pragma once

#include "dependent.cuh"
#include "rms.h"
#include "vec.cuh"

namespace dwconv {
namespace rms {

// V channels as stored, and their values
template <typename T, int V> struct Raw;
template <typename T> struct Raw<T, 1> { typedef T type; };
template <> struct Raw<float, 4> { typedef uint4 type; };
template <> struct Raw<__half, 8> { typedef uint4 type; };
template <> struct Raw<__nv_bfloat16, 8> { typedef uint4 type; };

template <typename T, int V>
__device__ __forceinline__ void widen(const typename Raw<T, V>::type& u, float* o) {
  if constexpr (V == 1) o[0] = to_f<T>(u);
  else unpack16<T>(u, o);
}
template <typename T, int V>
__device__ __forceinline__ typename Raw<T, V>::type narrow(const float* f) {
  if constexpr (V == 1) return from_f<T>(f[0]);
  else return pack16<T>(f);
}

inline bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// 16-byte vectors where every row of every tensor begins on 16 bytes
inline bool vec_ok(const Rms& g, int V, bool x, const void* codes) {
  return x && g.C % V == 0 && g.xs % V == 0 && g.xo % V == 0 && g.ys % V == 0 && g.yo % V == 0 &&
         reinterpret_cast<uintptr_t>(codes) % V == 0;
}

bool fwd_in_row(const Rms& g);  // rms.cu

}  // namespace rms
}  // namespace dwconv
