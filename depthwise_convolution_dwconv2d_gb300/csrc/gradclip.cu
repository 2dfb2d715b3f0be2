// Norm over all gradients of a model and their clipping:
//
//   n = sqrt(sum over all tensors of g^2),  k = min(1, most / (n + 1e-6)),  out = g * k
//
// The tensors' pointers travel in the kernels' parameters, so a call is two
// launches (per kBig tensors) whatever their number, and can be captured. The
// tensors are cut into units of kUnit elements; a block takes a run of
// neighbouring units, so it looks up its tensor once and then walks. The
// first launch leaves one sum of squares per block in the workspace; in the
// second every block adds those up in the same fixed order, and scales its
// units.
//
// Squares are added in fp32 over at most 256 elements, then in fp64. A square
// of fp32 or bf16 can be outside fp32's range where the value is not: a
// vector's sum that is not between 2^-90 and 2^110 (and does not come from
// zeros alone) is taken again in fp64, so no gradient of finite values has an
// infinite norm before n itself leaves fp32, and none vanishes.
//
// Bound by memory: each gradient is read once, read again (from L2, as far as
// it holds them: blocks walk their units backwards the second time) and
// written once.
#include <type_traits>

#include "dependent.cuh"
#include "gradclip.h"
#include "vec.cuh"

namespace dwconv {
namespace clip {
namespace {

constexpr int kNT = 256;
constexpr int kUnit = 4096;             // elements of a unit: 16 per thread
constexpr int64_t kBlocks = 152 * 8;    // what the GPU holds at once
constexpr int kSmall = 40, kBig = 960;  // tensors per launch: the parameters are 4 KB, or 32 KB, at most

template <int N>
struct Table {
  int count, units;
  int per_block;        // units of a block
  int slot0, slots;     // this launch's first partial sum; all launches' sums
  int first[N + 1];     // first unit of each tensor
  int dtype[N];
  const void* g[N];
  void* out[N];
  int64_t n[N];
};

template <int N>
__device__ __forceinline__ int tensor_of(const Table<N>& t, int unit) {
  int lo = 0, hi = t.count - 1;  // the last tensor whose first unit is at or before `unit`
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= unit) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ double squares_in_64(const float* v, int n) {
  double s = 0.0;
  for (int e = 0; e < n; ++e) s = fma((double)v[e], (double)v[e], s);
  return s;
}

// VEC values' squares into s, or into d where fp32 cannot hold them
template <typename T, int VEC>
__device__ __forceinline__ void add_squares(const float* v, float& s, double& d) {
  float a = 0.f, b = 0.f;
#pragma unroll
  for (int e = 0; e < VEC; e += 2) {
    a = fmaf(v[e], v[e], a);
    if (e + 1 < VEC) b = fmaf(v[e + 1], v[e + 1], b);
  }
  a += b;
  if (std::is_same<T, __half>::value) {
    s += a;  // fp16: squares lie between 2^-48 and 2^32
  } else if (a > 0x1p-90f && a < 0x1p110f) {
    s += a;
  } else {
    bool any = false;
#pragma unroll
    for (int e = 0; e < VEC; ++e) any |= v[e] != 0.f;
    if (any) d += squares_in_64(v, VEC);
  }
}

template <typename T>
__device__ __forceinline__ void unit_squares(const T* g, int64_t i0, int n, float& s, double& d) {
  constexpr int VEC = Vec<T>::n, K = kUnit / kNT / VEC;
  if (n == kUnit && reinterpret_cast<uintptr_t>(g) % 16 == 0) {
    uint4 u[K];
#pragma unroll
    for (int k = 0; k < K; ++k) u[k] = *reinterpret_cast<const uint4*>(g + i0 + ((int64_t)k * kNT + threadIdx.x) * VEC);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float v[VEC];
      unpack16<T>(u[k], v);
      add_squares<T, VEC>(v, s, d);
    }
  } else {
    for (int i = threadIdx.x; i < n; i += kNT) {
      const float v = to_f<T>(g[i0 + i]);
      add_squares<T, 1>(&v, s, d);
    }
  }
}

template <typename T>
__device__ __forceinline__ void unit_scale(const T* g, T* out, int64_t i0, int n, float k) {
  constexpr int VEC = Vec<T>::n, K = kUnit / kNT / VEC;
  if (n == kUnit && (reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(out)) % 16 == 0) {
    uint4 u[K];
#pragma unroll
    for (int q = 0; q < K; ++q) u[q] = *reinterpret_cast<const uint4*>(g + i0 + ((int64_t)q * kNT + threadIdx.x) * VEC);
#pragma unroll
    for (int q = 0; q < K; ++q) {
      float v[VEC];
      unpack16<T>(u[q], v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] *= k;
      *reinterpret_cast<uint4*>(out + i0 + ((int64_t)q * kNT + threadIdx.x) * VEC) = pack16<T>(v);
    }
  } else {
    for (int i = threadIdx.x; i < n; i += kNT) out[i0 + i] = from_f<T>(to_f<T>(g[i0 + i]) * k);
  }
}

__device__ __forceinline__ double block_sum(double d, double* sm) {
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = d;
  __syncthreads();
  d = 0.0;
#pragma unroll
  for (int w = 0; w < kNT / 32; ++w) d += sm[w];
  return d;
}

template <int N>
__global__ void __launch_bounds__(kNT)
squares_kernel(const __grid_constant__ Table<N> t, double* __restrict__ sums) {
  __shared__ double sm[kNT / 32];
  dependents_may_start();
  const int u0 = blockIdx.x * t.per_block;
  const int u1 = min(u0 + t.per_block, t.units);
  int q = tensor_of(t, u0);
  double d = 0.0;
  float s = 0.f;
  for (int u = u0; u < u1; ++u) {
    while (t.first[q + 1] <= u) ++q;
    const int64_t i0 = (int64_t)(u - t.first[q]) * kUnit;
    const int n = (int)min((int64_t)kUnit, t.n[q] - i0);
    DWCONV_DISPATCH_DTYPE(t.dtype[q], T, unit_squares((const T*)t.g[q], i0, n, s, d));
    if (((u - u0) & 15) == 15) {
      d += s;
      s = 0.f;
    }
  }
  d = block_sum(d + s, sm);
  if (threadIdx.x == 0) sums[t.slot0 + blockIdx.x] = d;
}

template <int N>
__global__ void __launch_bounds__(kNT)
scale_kernel(const __grid_constant__ Table<N> t, const double* __restrict__ sums, float most, float* norm) {
  __shared__ double sm[kNT / 32];
  const int u0 = blockIdx.x * t.per_block;
  const int u1 = min(u0 + t.per_block, t.units);
  wait_for_previous();
  double d = 0.0;
  for (int i = threadIdx.x; i < t.slots; i += kNT) d += sums[i];
  const double n = sqrt(block_sum(d, sm));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0 && t.slot0 == 0) *norm = (float)n;
  const double c = isinf(most) ? 1.0 : (double)most / (n + 1e-6);
  const float k = c >= 1.0 ? 1.f : (float)c;  // NaN stays
  if (u1 <= u0) return;
  int q = tensor_of(t, u1 - 1);
  for (int u = u1 - 1; u >= u0; --u) {
    while (t.first[q] > u) --q;
    void* const out = t.out[q];
    if (!out || (k == 1.f && out == t.g[q])) continue;
    const int64_t i0 = (int64_t)(u - t.first[q]) * kUnit;
    const int m = (int)min((int64_t)kUnit, t.n[q] - i0);
    DWCONV_DISPATCH_DTYPE(t.dtype[q], T, unit_scale((const T*)t.g[q], (T*)out, i0, m, k));
  }
}

int64_t units_of(int64_t n) { return (n + kUnit - 1) / kUnit; }

// Runs of tensors that one launch takes: at most kBig of them and 2^30 units.
// fn(first, count of tensors, units)
template <typename F>
cudaError_t over_launches(int count, const dwconv_grad_t* grads, F fn) {
  int i = 0;
  while (i < count) {
    int used = 0, j = i;
    int64_t units = 0;
    for (; j < count && used < kBig; ++j) {
      const int64_t u = units_of(grads[j].n);
      if (u == 0) continue;
      if (used > 0 && units + u > (int64_t(1) << 30)) break;
      units += u;
      ++used;
    }
    if (used > 0) {
      const cudaError_t e = fn(i, j, used, units);
      if (e != cudaSuccess) return e;
    }
    i = j;
  }
  return cudaSuccess;
}

int blocks_of(int64_t units) {
  const int64_t per = (units + kBlocks - 1) / kBlocks;
  return (int)((units + per - 1) / per);
}

template <int N>
cudaError_t launch(const dwconv_grad_t* grads, int i, int j, int64_t units, int slot0, int slots, bool scale, float most,
                   float* norm, double* sums, cudaStream_t s) {
  Table<N> t;
  t.count = 0;
  t.units = (int)units;
  const int blocks = blocks_of(units);
  t.per_block = (int)((units + blocks - 1) / blocks);
  t.slot0 = slot0;
  t.slots = slots;
  int64_t u = 0;
  for (; i < j; ++i) {
    if (grads[i].n == 0) continue;
    t.first[t.count] = (int)u;
    t.dtype[t.count] = grads[i].dtype;
    t.g[t.count] = grads[i].g;
    t.out[t.count] = grads[i].out;
    t.n[t.count] = grads[i].n;
    u += units_of(grads[i].n);
    ++t.count;
  }
  t.first[t.count] = (int)u;
  if (!scale) {
    squares_kernel<N><<<blocks, kNT, 0, s>>>(t, sums);
    return cudaGetLastError();
  }
  return launch_dependent(scale_kernel<N>, dim3(blocks), dim3(kNT), 0, s, t, (const double*)sums, most, norm);
}

__global__ void no_gradients_kernel(float* norm) { *norm = 0.f; }

}  // namespace

size_t workspace_bytes(int count, const dwconv_grad_t* grads) {
  int64_t slots = 0;
  over_launches(count, grads, [&](int, int, int, int64_t units) {
    slots += blocks_of(units);
    return cudaSuccess;
  });
  return (size_t)slots * sizeof(double);
}

cudaError_t run(int count, const dwconv_grad_t* grads, float most, float* norm, void* ws, cudaStream_t s) {
  double* sums = (double*)ws;
  const int slots = (int)(workspace_bytes(count, grads) / sizeof(double));
  if (slots == 0) {
    if (!norm) return cudaSuccess;
    no_gradients_kernel<<<1, 1, 0, s>>>(norm);
    return cudaGetLastError();
  }
  cudaError_t e = cudaSuccess;
  for (int scale = 0; scale < 2 && e == cudaSuccess; ++scale) {
    int slot0 = 0;
    e = over_launches(count, grads, [&](int i, int j, int used, int64_t units) {
      const cudaError_t r = used <= kSmall
                                ? launch<kSmall>(grads, i, j, units, slot0, slots, scale != 0, most, norm, sums, s)
                                : launch<kBig>(grads, i, j, units, slot0, slots, scale != 0, most, norm, sums, s);
      slot0 += blocks_of(units);
      return r;
    });
  }
  return e;
}

}  // namespace clip
}  // namespace dwconv
