// Norm over all gradients of a model and their clipping:
//
//   n = sqrt(sum over all tensors of g^2),  k = min(1, most / (n + 1e-6)),  out = g * k
//
// The tensors' pointers travel in the kernels' parameters, so a call is two
// launches (per kBig tensors) whatever their number, and can be captured. The
// tensors are cut into units of kUnit elements; a warp takes a run of
// neighbouring units, so it looks up its tensor once and then walks. The first
// launch leaves one sum of squares per block in the workspace; in the second
// every block adds those up in the same fixed order, and scales its units.
// Where one cluster of blocks can take all units, it does both in one launch
// and joins its sums through its shared memory.
//
// Squares are added in fp32 over at most 256 elements of a thread and 32
// threads, then in fp64: as seldom as that because the GPU adds two fp64 a
// clock and SM (with every thread joining in fp64, and the root and quotient
// by every thread, 91 tensors of 6.4 MB took 33 us). A square of fp32 or bf16
// can be outside fp32's range where the value is not: a vector's sum that is
// not between 2^-90 and 2^110 (and does not come from zeros alone) is taken
// again in fp64, so no gradient of finite values has an infinite norm before
// n itself leaves fp32, and none vanishes. The root and the quotient are
// fp32: the sum's rounding, halved by the root, the root's, that of n + 1e-6
// and the quotient's put the factor within 3.5 * 2^-24 of itself (1 if it came
// from fp64, of which an SM makes two a clock). The output's own rounding
// follows: nothing beside it in 16 bits.
//
// Bound by memory: each gradient is read once, read again (from L2, as far as
// it holds them: warps walk their units backwards the second time) and
// written once.
#include <type_traits>

#include <cooperative_groups.h>

#include "dependent.cuh"
#include "gradclip.h"
#include "vec.cuh"

namespace dwconv {
namespace clip {
namespace {

namespace cg = cooperative_groups;

constexpr int kNT = 512, kWarps = kNT / 32;
constexpr int kUnit = 512;              // elements of a unit: 16 per lane
constexpr int64_t kBlocks = 152 * 4;    // what the GPU holds at once
constexpr int kCluster = 8;             // blocks of a cluster
// Units that one cluster takes by itself: one a warp. fp32, 4 tensors, in one
// launch against two, back to back in a graph / whole calls with a cold L2, us:
// 2820 elements 4.6 / 16.3 against 5.0 / 20.9; 65536 5.4 / 16.2 against 5.7 /
// 19.5; 131072 6.9 / 18.1 against 5.9 / 19.8; 262144 9.2 / 21.8 against 5.7 /
// 20.1; 524288 14.3 / 28.1 against 6.2 / 19.5. 100 tensors: 65536 7.7 / 21.0
// against 6.4 / 22.4, 131072 8.9 / 22.6 against 6.8 / 22.3.
constexpr int kAlone = kCluster * kWarps;
// Tensors per launch, by sizes of the parameters (1.3 to 31 KB): a launch with
// 31 KB of them takes 6 us longer than one with 4.
constexpr int kSmall = 40, kMid = 120, kMore = 240, kMany = 480, kBig = 960;

template <int N>
struct Table {
  int count, units;
  int per_warp;         // units of a warp
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
    s += a;  // squares lie between 2^-48 and 2^32
  } else if (a > 0x1p-90f && a < 0x1p110f) {
    s += a;
  } else {
    bool any = false;
#pragma unroll
    for (int e = 0; e < VEC; ++e) any |= v[e] != 0.f;
    if (any) d += squares_in_64(v, VEC);
  }
}

// A unit of n elements: whole 16-byte vectors where its pointers allow it,
// the elements behind them (or all, off 16 bytes) one by one. A lane's vectors
// are on their way before the first is used.
template <typename T>
__device__ __forceinline__ void unit_squares(const T* g, int n, float& s, double& d) {
  constexpr int VEC = Vec<T>::n, K = kUnit / 32 / VEC;
  const int lane = threadIdx.x & 31;
  if (reinterpret_cast<uintptr_t>(g) % 16 == 0) {
    uint4 u[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      u[k] = make_uint4(0, 0, 0, 0);
      if ((k * 32 + lane + 1) * VEC <= n) u[k] = reinterpret_cast<const uint4*>(g)[k * 32 + lane];
    }
    const int rest = n % VEC;
    float v[VEC];
    if (lane < rest) {
      v[0] = to_f<T>(g[n - rest + lane]);
      add_squares<T, 1>(v, s, d);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      unpack16<T>(u[k], v);
      add_squares<T, VEC>(v, s, d);
    }
  } else {
#pragma unroll 1
    for (int i = lane; i < n; i += 128) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = i + 32 * k < n ? to_f<T>(g[i + 32 * k]) : 0.f;
      add_squares<T, 4>(v, s, d);
    }
  }
}

template <typename T>
__device__ __forceinline__ uint4 times(const uint4& u, float k) {
  constexpr int VEC = Vec<T>::n;
  float v[VEC];
  unpack16<T>(u, v);
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] *= k;
  return pack16<T>(v);
}
template <typename T>
__device__ __forceinline__ void unit_scale(const T* g, T* out, int n, float k) {
  constexpr int VEC = Vec<T>::n, K = kUnit / 32 / VEC;
  const int lane = threadIdx.x & 31;
  if ((reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(out)) % 16 == 0) {
    const uint4* from = reinterpret_cast<const uint4*>(g) + lane;
    uint4* to = reinterpret_cast<uint4*>(out) + lane;
    if (n == kUnit) {
      uint4 u[K];
#pragma unroll
      for (int q = 0; q < K; ++q) u[q] = from[q * 32];
#pragma unroll
      for (int q = 0; q < K; ++q) to[q * 32] = times<T>(u[q], k);
      return;
    }
    const int whole = n / VEC;
#pragma unroll 2
    for (int q = lane; q < whole; q += 32, from += 32, to += 32) *to = times<T>(*from, k);
    const int i = whole * VEC + lane;
    if (i < n) out[i] = from_f<T>(to_f<T>(g[i]) * k);
  } else {
#pragma unroll 4
    for (int i = lane; i < n; i += 32) out[i] = from_f<T>(to_f<T>(g[i]) * k);
  }
}

// All threads' sums, in thread 0 of a block of kNT threads
__device__ __forceinline__ double block_sum(float s, double d, double* sm) {
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (__any_sync(0xffffffffu, d != 0.0))  // NaN counts
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = d + (double)s;
  __syncthreads();
  double t = 0.0;
  if (threadIdx.x == 0)
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t += sm[w];
  return t;
}

// sum of squares -> n and k, in fp32 but for the sum's range
__device__ __forceinline__ float factor_of(double sum, float most, float* n) {
  // sum = m * 4^e with m in [1, 4): fp32 holds m's root times 2^e wherever it holds n
  const int e = sum > 0.0 && sum < 1.7e308 ? (((__double2hiint(sum) >> 20) & 0x7ff) - 1023) >> 1 : 0;
  const double m = __hiloint2double(__double2hiint(sum) - e * (1 << 21), __double2loint(sum));
  *n = scalbnf(__fsqrt_rn((float)m), e);
  if (isinf(most)) return 1.f;
  const float c = __fdiv_rn(most, *n + 1e-6f);
  return c >= 1.f ? 1.f : c;  // NaN stays
}

// The units of this warp: u0 <= u < u1
template <int N>
__device__ __forceinline__ void run_of(const Table<N>& t, int& u0, int& u1) {
  u0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * t.per_warp;
  u1 = min(u0 + t.per_warp, t.units);
}

template <int N>
__device__ __forceinline__ void sum_units(const Table<N>& t, int u0, int u1, float& s, double& d) {
  if (u0 >= u1) return;
  int q = tensor_of(t, u0);
  for (int u = u0; u < u1; ++u) {
    while (t.first[q + 1] <= u) ++q;
    const int64_t i0 = (int64_t)(u - t.first[q]) * kUnit;
    const int n = (int)min((int64_t)kUnit, t.n[q] - i0);
    DWCONV_DISPATCH_DTYPE(t.dtype[q], T, unit_squares((const T*)t.g[q] + i0, n, s, d));
    if (((u - u0) & 15) == 15) {
      d += s;
      s = 0.f;
    }
  }
}
template <int N>
__device__ __forceinline__ void scale_units(const Table<N>& t, int u0, int u1, float k) {
  if (u0 >= u1) return;
  int q = tensor_of(t, u1 - 1);
  for (int u = u1 - 1; u >= u0; --u) {
    while (t.first[q] > u) --q;
    void* const out = t.out[q];
    if (!out || (k == 1.f && out == t.g[q])) continue;
    const int64_t i0 = (int64_t)(u - t.first[q]) * kUnit;
    const int n = (int)min((int64_t)kUnit, t.n[q] - i0);
    DWCONV_DISPATCH_DTYPE(t.dtype[q], T, unit_scale((const T*)t.g[q] + i0, (T*)out + i0, n, k));
  }
}

template <int N>
__global__ void __launch_bounds__(kNT)
squares_kernel(const __grid_constant__ Table<N> t, double* __restrict__ sums) {
  __shared__ double sm[kWarps];
  dependents_may_start();
  int u0, u1;
  run_of(t, u0, u1);
  double d = 0.0;
  float s = 0.f;
  sum_units(t, u0, u1, s, d);
  d = block_sum(s, d, sm);
  if (threadIdx.x == 0) sums[t.slot0 + blockIdx.x] = d;
}

template <int N>
__global__ void __launch_bounds__(kNT)
scale_kernel(const __grid_constant__ Table<N> t, const double* __restrict__ sums, float most, float* norm) {
  __shared__ float factor;
  int u0, u1;
  run_of(t, u0, u1);
  wait_for_previous();
  if (threadIdx.x < 32) {
    double d = 0.0;
#pragma unroll 4
    for (int i = threadIdx.x; i < t.slots; i += 32) d += sums[i];
    for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (threadIdx.x == 0) {
      float n;
      factor = factor_of(d, most, &n);
      if (norm && blockIdx.x == 0 && t.slot0 == 0) *norm = n;
    }
  }
  __syncthreads();
  scale_units(t, u0, u1, factor);
}

// Both in one launch of one cluster.
template <int N>
__global__ void __launch_bounds__(kNT)
alone_kernel(const __grid_constant__ Table<N> t, float most, float* norm) {
  __shared__ double sm[kWarps], mine;
  __shared__ float factor;
  cg::cluster_group cl = cg::this_cluster();
  int u0, u1;
  run_of(t, u0, u1);
  double d = 0.0;
  float s = 0.f;
  sum_units(t, u0, u1, s, d);
  d = block_sum(s, d, sm);
  if (threadIdx.x == 0) mine = d;
  cl.sync();
  if (threadIdx.x == 0) {
    double all = 0.0;
    for (unsigned k = 0; k < gridDim.x; ++k) all += *cl.map_shared_rank(&mine, k);
    float n;
    factor = factor_of(all, most, &n);
    if (norm && blockIdx.x == 0) *norm = n;
  }
  cl.sync();  // and no block leaves while others read its sum
  scale_units(t, u0, u1, factor);
}

__global__ void no_gradients_kernel(float* norm) { *norm = 0.f; }

// ---- host -----------------------------------------------------------------------

int64_t units_of(int64_t n) { return (n + kUnit - 1) / kUnit; }

// Runs of tensors that one launch takes, kBig of them at most.
// fn(first, end, tensors with elements, units)
template <typename F>
cudaError_t over_launches(int count, const dwconv_grad_t* grads, F fn) {
  for (int i = 0; i < count;) {
    int used = 0, j = i;
    int64_t units = 0;
    for (; j < count && used < kBig; ++j) {
      units += units_of(grads[j].n);
      used += grads[j].n > 0;
    }
    if (used > 0) {
      const cudaError_t e = fn(i, j, used, units);
      if (e != cudaSuccess) return e;
    }
    i = j;
  }
  return cudaSuccess;
}

int per_warp_of(int64_t units, int64_t most) { return (int)((units + most * kWarps - 1) / (most * kWarps)); }
int blocks_of(int64_t units, int64_t most = kBlocks) {
  const int64_t per = (int64_t)per_warp_of(units, most) * kWarps;
  return (int)((units + per - 1) / per);
}

// Tensors i .. j - 1, as the warps of at most `most` blocks take them
template <int N>
void fill(Table<N>& t, const dwconv_grad_t* grads, int i, int j, int64_t units, int64_t most, int slot0, int slots) {
  t.count = 0;
  t.units = (int)units;
  t.per_warp = per_warp_of(units, most);
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
}

template <int N>
cudaError_t launch(const dwconv_grad_t* grads, int i, int j, int64_t units, int slot0, int slots, bool scale, float most,
                   float* norm, double* sums, cudaStream_t s) {
  Table<N> t;
  const int blocks = blocks_of(units);
  fill(t, grads, i, j, units, kBlocks, slot0, slots);
  if (!scale) {
    squares_kernel<N><<<blocks, kNT, 0, s>>>(t, sums);
    return cudaGetLastError();
  }
  return launch_dependent(scale_kernel<N>, dim3(blocks), dim3(kNT), 0, s, t, (const double*)sums, most, norm);
}

template <int N>
cudaError_t launch_alone(const dwconv_grad_t* grads, int i, int j, int64_t units, float most, float* norm, cudaStream_t s) {
  Table<N> t;
  const int blocks = blocks_of(units, kCluster);
  fill(t, grads, i, j, units, kCluster, 0, 0);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)blocks;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kNT);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, alone_kernel<N>, t, most, norm);
  return e != cudaSuccess ? e : cudaGetLastError();
}

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
  int launches = 0, slots = 0;
  over_launches(count, grads, [&](int, int, int, int64_t units) {
    slots += blocks_of(units);
    ++launches;
    return cudaSuccess;
  });
  if (launches == 0) {
    if (!norm) return cudaSuccess;
    no_gradients_kernel<<<1, 1, 0, s>>>(norm);
    return cudaGetLastError();
  }
  cudaError_t e = cudaSuccess;
  for (int scale = 0; scale < 2 && e == cudaSuccess; ++scale) {
    int slot0 = 0;
    e = over_launches(count, grads, [&](int i, int j, int used, int64_t units) {
      if (launches == 1 && units <= kAlone && used <= kMid)
        return scale ? cudaSuccess
               : used <= kSmall ? launch_alone<kSmall>(grads, i, j, units, most, norm, s)
                                : launch_alone<kMid>(grads, i, j, units, most, norm, s);
      auto* const go = used <= kSmall ? launch<kSmall> : used <= kMid ? launch<kMid> : used <= kMore ? launch<kMore>
                       : used <= kMany ? launch<kMany> : launch<kBig>;
      const cudaError_t r = go(grads, i, j, units, slot0, slots, scale != 0, most, norm, sums, s);
      slot0 += blocks_of(units);
      return r;
    });
  }
  return e;
}

}  // namespace clip
}  // namespace dwconv
