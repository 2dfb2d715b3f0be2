// Helpers shared by the RMS norm's forward and backward kernels.
#pragma once

#include "dependent.cuh"
#include "f32x2.cuh"
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

// ---- rows that begin anywhere ---------------------------------------------------
// A row whose first channel lies `ph` elements behind a 16-byte boundary is
// read in the vectors that lie on 16 bytes: vector v holds the channels cb =
// v * V - ph and on. The first and last ones reach over the row's ends: their
// elements outside it belong to rows before and after it (or to what lies
// between two rows), are read with the vector while that lies within the
// tensor, count as zeros and are not written. Rows a multiple of 8 apart begin
// alike, so a thread that steps over rows that far keeps its channels.

// Rows whose vectors lie within the tensor: no vector reaches over 8 elements.
__device__ __forceinline__ bool inner_row(int64_t row, int64_t rows) { return row >= 8 && row < rows - 8; }

// element by element
template <typename T, int V>
__device__ __forceinline__ typename Raw<T, V>::type load_part(const T* row, int cb, int C) {
  alignas(16) T v[V];
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = cb + e >= 0 && cb + e < C ? row[cb + e] : from_f<T>(0.f);
  return *reinterpret_cast<const typename Raw<T, V>::type*>(v);
}
// zeros in place of the elements outside the row
template <typename T, int V>
__device__ __forceinline__ void clear_part(typename Raw<T, V>::type& u, int cb, int C) {
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (V == 4) {
      if (cb + j < 0 || cb + j >= C) w[j] = 0;
    } else {
      if (cb + 2 * j < 0 || cb + 2 * j >= C) w[j] &= 0xffff0000u;
      if (cb + 2 * j + 1 < 0 || cb + 2 * j + 1 >= C) w[j] &= 0xffffu;
    }
  }
}
template <typename T, int V, bool RAG>
__device__ __forceinline__ typename Raw<T, V>::type load_ends(const T* row, int cb, int C) {
  if constexpr (RAG) return load_part<T, V>(row, cb, C);
  else return *reinterpret_cast<const typename Raw<T, V>::type*>(row + cb);
}
// The elements of a vector over one of the row's ends, in pieces of 8, 4 and 2
// bytes; over both, element by element.
template <typename T, int V>
__device__ __forceinline__ void store_part(T* row, int cb, int C, const typename Raw<T, V>::type& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  char* at = reinterpret_cast<char*>(row + cb);
  if (cb < 0 && cb + V > C) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (cb + e < 0 || cb + e >= C) continue;
      if constexpr (V == 4) *reinterpret_cast<uint32_t*>(at + 4 * e) = w[e];
      else *reinterpret_cast<uint16_t*>(at + 2 * e) = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
    }
    return;
  }
  constexpr int es = sizeof(T);
  if (cb < 0) {  // the last m elements
    const int m = V + cb;
    if (m & (8 / es)) *reinterpret_cast<uint2*>(at + 8) = make_uint2(w[2], w[3]);
    const uint32_t x = m & (8 / es) ? w[1] : w[3];
    if (m & (4 / es)) *reinterpret_cast<uint32_t*>(at + 16 - (m & (12 / es)) * es) = x;
    if constexpr (es == 2) {
      const uint32_t z = m & 2 ? (m & 4 ? w[0] : w[2]) : x;
      if (m & 1) *reinterpret_cast<uint16_t*>(at + 16 - m * 2) = (uint16_t)(z >> 16);
    }
  } else {  // the first m
    const int m = C - cb;
    if (m & (8 / es)) *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
    const uint32_t x = m & (8 / es) ? w[2] : w[0];
    if (m & (4 / es)) *reinterpret_cast<uint32_t*>(at + (m & (8 / es)) * es) = x;
    if constexpr (es == 2) {
      const uint32_t z = m & 2 ? (m & 4 ? w[3] : w[1]) : x;
      if (m & 1) *reinterpret_cast<uint16_t*>(at + (m & 6) * 2) = (uint16_t)z;
    }
  }
}
template <typename T, int V, bool RAG>
__device__ __forceinline__ void store_vec(T* row, int cb, int C, const typename Raw<T, V>::type& u) {
  if (RAG && (cb < 0 || cb + V > C)) store_part<T, V>(row, cb, C, u);
  else *reinterpret_cast<typename Raw<T, V>::type*>(row + cb) = u;
}
// elements between the 16-byte boundary before p and p
template <typename T>
__device__ __forceinline__ int phase_of(const T* p) { return (int)(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(T)); }

// pairs of a vector's values, and back with one rounding
template <typename T, int V>
__device__ __forceinline__ void pairs_of(const typename Raw<T, V>::type& u, f32x2* o) { unpack16_pairs<T>(u, o); }
template <typename T, int V>
__device__ __forceinline__ typename Raw<T, V>::type vec_of(const f32x2* p) {
  float f[V];
#pragma unroll
  for (int e = 0; e < V / 2; ++e) unpack_f32x2(p[e], f[2 * e], f[2 * e + 1]);
  return pack16<T>(f);
}

__device__ __forceinline__ f32x2 both(float v) { return pack_f32x2(v, v); }
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  fma_f32x2(c, a, b);
  return c;
}
__device__ __forceinline__ float sum2(f32x2 v) {
  float a, b;
  unpack_f32x2(v, a, b);
  return a + b;
}

// A row's sum, in all of its tpr threads. part: NT / 32 values of shared
// memory, not written again before another barrier.
template <int NT>
__device__ __forceinline__ float row_sum(float s, int tpr, float* part) {
  const int tid = threadIdx.x, lane = tid & 31;
  if (tpr >= 32) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  } else {
    for (int o = tpr >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  }
  if (tpr > 32) {
    if (lane == 0) part[tid >> 5] = s;
    __syncthreads();
    const int nw = tpr >> 5, w0 = (tid >> 5) & ~(nw - 1);
    if (NT <= 256) {  // eight warps at most: read all of the row's
      s = 0.f;
#pragma unroll
      for (int w = 0; w < NT / 32; ++w) s += w < nw ? part[w0 + w] : 0.f;
    } else {
      s = lane < nw ? part[w0 + lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    }
  }
  return s;
}

inline bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// 16-byte vectors where every row of every tensor begins on 16 bytes (`all` of
// the pointers do); vectors over the ends where all of them begin alike.
inline bool rows_on16(const Rms& g, int V) {
  return g.C % V == 0 && g.xs % V == 0 && g.xo % V == 0 && g.ys % V == 0 && g.yo % V == 0;
}
inline bool rows_alike(const Rms& g, int V) { return (g.xs - g.ys) % V == 0 && (g.xo - g.yo) % V == 0; }
inline bool alike(const void* a, const void* b) {
  return !a || !b || (reinterpret_cast<uintptr_t>(a) - reinterpret_cast<uintptr_t>(b)) % 16 == 0;
}

bool fwd_in_row(const Rms& g);  // rms.cu

}  // namespace rms
}  // namespace dwconv
