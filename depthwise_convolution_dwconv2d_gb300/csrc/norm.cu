// Channels-last group norm with an activation, forward and backward: plans,
// dispatch, and the split kernels, for the shapes that the slab and stream
// kernels (norm_slab_impl.cuh) leave: slices wider than a block, that is
// groups of more than 1024 channels (2048 in aligned 16-bit rows, but for a
// backward that reads x in full: it takes four channels per thread, and past
// 1024 runs here with one, 89 us at 8x32x32x1536 bf16 in one group).
//
// A sample's group is spread over C / D channels of every pixel, so its sums
// need all of the sample before the first output. Here that is two reads of
// the inputs with a small reduction between them:
//
//  1. partial sums per (sample, chunk of pixels, channel), one thread per
//     vector of channels and row lane, the row lanes joined in shared memory;
//  2. one block per (sample, group) joins chunks and channels, in index order;
//  3. the inputs again, and the outputs; forward chunks run last to first, so
//     that the second read begins with what the first left in L2.
//
// The variance is not taken from sums of squares of x: a thread sums
// (x - s) and (x - s)^2 with s its own first value of the channel, turns
// them into a mean and a sum of squares about that mean, and these are joined
// by the parallel form of the two (Chan, Golub and LeVeque, "Updating
// formulae and a pairwise algorithm for computing sample variances", 1979).
// All sums are fp32; every order is fixed, so results are bit-reproducible.
#include "norm.cuh"
#include "norm_slab.h"

namespace dwconv {
namespace norm {
namespace {

constexpr int kNT = 256;

// Rows that a thread adds up one after another, as far as chunks go. A chain of n fp32 additions of like terms can be off
// by n / 4 * 2^-24 of the sum (constant terms), so samples that would fill the GPU with a long chunk each are cut too.
constexpr int64_t kChain = 4096;

// How the split kernels cut a sample: channels into slices of tc vectors,
// pixels into chunks.
struct Cut {
  int tc;          // vectors of channels per slice (a power of two)
  int rl;          // row lanes: kNT / tc
  int slices, chunks;
  int64_t rows;    // pixels per chunk
  int64_t units;   // N * chunks * slices
};

Cut plan_cut(const Norm& g, int V) {
  Cut k{};
  const int vecs = (g.C + V - 1) / V;
  k.tc = V == 1 ? 32 : 16;
  while (k.tc > 1 && k.tc / 2 >= vecs) k.tc /= 2;
  k.rl = kNT / k.tc;
  k.slices = (vecs + k.tc - 1) / k.tc;
  // enough blocks to fill the GPU a few times over, chunks of at least 4 rows per row lane
  int64_t want = (152 * 8 + g.N * k.slices - 1) / (g.N * k.slices);
  const int64_t chains = (g.P + kChain * k.rl - 1) / (kChain * k.rl), most = (g.P + 4 * k.rl - 1) / (4 * k.rl);
  if (want < chains) want = chains;
  if (want > most) want = most;
  if (want > 256) want = 256;
  if (want < 1) want = 1;
  k.rows = (g.P + want - 1) / want;
  k.chunks = (int)((g.P + k.rows - 1) / k.rows);
  k.units = g.N * k.chunks * (int64_t)k.slices;
  return k;
}

struct Unit {
  int64_t n, r0, r1;
  int chunk, c;   // first channel of this thread's vector, or C where it has none
  int rl;
};

template <int V>
__device__ __forceinline__ Unit unit_of(const Norm& g, const Cut& k, int64_t u) {
  Unit w;
  const int slice = (int)(u % k.slices);
  u /= k.slices;
  w.chunk = (int)(u % k.chunks);
  w.n = u / k.chunks;
  w.r0 = w.chunk * k.rows;
  w.r1 = min(w.r0 + k.rows, g.P);
  w.c = min((slice * k.tc + (int)(threadIdx.x & (k.tc - 1))) * V, g.C);
  w.rl = threadIdx.x / k.tc;
  return w;
}

// Sums `v` over the row lanes, in lane order; the sum goes to lane 0's thread.
template <int V>
__device__ __forceinline__ void join_rows(const Cut& k, float* sm, float* v) {
#pragma unroll
  for (int e = 0; e < V; ++e) sm[e * kNT + threadIdx.x] = v[e];
  __syncthreads();
  if (threadIdx.x < k.tc) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float a = 0.f;
      for (int r = 0; r < k.rl; ++r) a += sm[e * kNT + r * k.tc + threadIdx.x];
      sm[e * kNT + threadIdx.x] = a;
    }
  }
  __syncthreads();
  const int t = threadIdx.x & (k.tc - 1);
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = sm[e * kNT + t];
  __syncthreads();
}

// part[n][chunk][c] = (mean, sum of squares about it) of the chunk's rows
template <typename T, int V>
__global__ void __launch_bounds__(kNT)
moments_kernel(Norm g, Cut k, const T* __restrict__ x, float2* __restrict__ part) {
  __shared__ float sm[kNT * V];
  for (int64_t u = blockIdx.x; u < k.units; u += gridDim.x) {
    const Unit w = unit_of<V>(g, k, u);
    float s[V], d[V], q[V];
    int cnt = 0;
#pragma unroll
    for (int e = 0; e < V; ++e) s[e] = d[e] = q[e] = 0.f;
    if (w.c < g.C) {
      const T* p = x + (w.n * g.P) * g.xs + g.xo + w.c;
      int64_t r = w.r0 + w.rl;
      if (r < w.r1) load_v<T, V>(p + r * g.xs, s);
#pragma unroll 4
      for (; r < w.r1; r += k.rl) {
        float f[V];
        load_v<T, V>(p + r * g.xs, f);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float t = f[e] - s[e];
          d[e] += t;
          q[e] = fmaf(t, t, q[e]);
        }
        ++cnt;
      }
    }
    // the thread's mean and squares about it, then about the chunk's mean
    const float inv = cnt > 0 ? 1.f / (float)cnt : 0.f;
    float m[V], a[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      m[e] = s[e] + d[e] * inv;
      const float t = q[e] - d[e] * d[e] * inv;
      q[e] = t < 0.f ? 0.f : t;  // NaN stays
      a[e] = (float)cnt * m[e];
    }
    join_rows<V>(k, sm, a);
    const float rows = (float)(w.r1 - w.r0);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      a[e] /= rows;
      const float t = m[e] - a[e];
      q[e] += (float)cnt * t * t;
    }
    join_rows<V>(k, sm, q);
    if (w.rl == 0 && w.c < g.C) {
      float2* o = part + (w.n * k.chunks + w.chunk) * g.C + w.c;
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = make_float2(a[e], q[e]);
    }
  }
}

// sum over the block, in a fixed order
__device__ __forceinline__ float block_sum(float v, float* sm) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  float a = 0.f;
  for (int i = 0; i < (int)blockDim.x / 32; ++i) a += sm[i];
  __syncthreads();
  return a;
}

// stats[n][g] = (mean, rstd) from the chunks' moments
__global__ void __launch_bounds__(kNT)
group_moments_kernel(Norm g, Cut k, const float2* __restrict__ part, float2* __restrict__ stats,
                     float* __restrict__ mean_out, float* __restrict__ rstd_out) {
  __shared__ float sm[kNT / 32];
  for (int64_t i = blockIdx.x; i < g.N * g.G; i += gridDim.x) {
    const int64_t n = i / g.G;
    const int c0 = (int)(i - n * g.G) * g.D;
    const int64_t entries = (int64_t)k.chunks * g.D;
    float a = 0.f;
    for (int64_t j = threadIdx.x; j < entries; j += kNT) {
      const int64_t ch = j / g.D;
      const float rows = (float)(min((ch + 1) * k.rows, g.P) - ch * k.rows);
      a = fmaf(rows, part[(n * k.chunks + ch) * g.C + c0 + (j - ch * g.D)].x, a);
    }
    const float total = (float)g.P * (float)g.D;
    const float mean = block_sum(a, sm) / total;
    float q = 0.f;
    for (int64_t j = threadIdx.x; j < entries; j += kNT) {
      const int64_t ch = j / g.D;
      const float rows = (float)(min((ch + 1) * k.rows, g.P) - ch * k.rows);
      const float2 p = part[(n * k.chunks + ch) * g.C + c0 + (j - ch * g.D)];
      const float t = p.x - mean;
      q += fmaf(rows * t, t, p.y);
    }
    q = block_sum(q, sm);
    if (threadIdx.x == 0) {
      const float rstd = 1.f / sqrtf(q / total + g.eps);
      stats[i] = make_float2(mean, rstd);
      if (mean_out) mean_out[i] = mean;
      if (rstd_out) rstd_out[i] = rstd;
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void load_affine(const Norm& g, int c, const T* gamma, const T* beta, float* ga,
                                            float* be) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
    ga[e] = gamma ? ld(gamma + c + e) : 1.f;
    be[e] = beta ? ld(beta + c + e) : 0.f;
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kNT)
apply_kernel(Norm g, Cut k, const T* __restrict__ x, const T* __restrict__ gamma, const T* __restrict__ beta,
             const float2* __restrict__ stats, T* __restrict__ y) {
  for (int64_t i = blockIdx.x; i < k.units; i += gridDim.x) {
    const Unit w = unit_of<V>(g, k, k.units - 1 - i);
    if (w.c >= g.C) continue;
    float ga[V], be[V], mu[V], rs[V];
    load_affine<T, V>(g, w.c, gamma, beta, ga, be);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float2 st = stats[w.n * g.G + (w.c + e) / g.D];
      mu[e] = st.x;
      rs[e] = st.y;
    }
    const T* p = x + (w.n * g.P) * g.xs + g.xo + w.c;
    T* o = y + (w.n * g.P) * g.ys + g.yo + w.c;
#pragma unroll 4
    for (int64_t r = w.r0 + w.rl; r < w.r1; r += k.rl) {
      float f[V];
      load_v<T, V>(p + r * g.xs, f);
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = affine(xhat(f[e], mu[e], rs[e]), ga[e], be[e]);
      act_v<V>(g.act, f);
      store_v<T, V>(o + r * g.ys, f);
    }
  }
}

// The input of the backward: the storage type or a checkpoint.
template <typename T, int SRC, int V>
__device__ __forceinline__ void load_src(const Norm& g, const T* x, const Act8& t, int64_t row, int c, float* f) {
  if constexpr (SRC == kSrcFull) {
    load_v<T, V>(x + row * g.xs + g.xo + c, f);
  } else {
    load_act8<SRC, V>(t, row, g.C, c, f);
  }
}

// part[n][chunk][c] = (sum du, sum du * xh) over the chunk's rows
template <typename T, int SRC, int V>
__global__ void __launch_bounds__(kNT)
grad_sums_kernel(Norm g, Cut k, const T* __restrict__ x, Act8 x8, const T* __restrict__ gy,
                 const T* __restrict__ gamma, const T* __restrict__ beta, const float* __restrict__ mean,
                 const float* __restrict__ rstd, float2* __restrict__ part) {
  __shared__ float sm[kNT * V];
  for (int64_t u = blockIdx.x; u < k.units; u += gridDim.x) {
    const Unit w = unit_of<V>(g, k, u);
    float a[V], b[V];
#pragma unroll
    for (int e = 0; e < V; ++e) a[e] = b[e] = 0.f;
    if (w.c < g.C) {
      float ga[V], be[V], mu[V], rs[V];
      load_affine<T, V>(g, w.c, gamma, beta, ga, be);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int64_t at = w.n * g.G + (w.c + e) / g.D;
        mu[e] = __ldg(mean + at);
        rs[e] = __ldg(rstd + at);
      }
#pragma unroll 2
      for (int64_t r = w.r0 + w.rl; r < w.r1; r += k.rl) {
        const int64_t row = w.n * g.P + r;
        float f[V], d[V], t[V];
        load_src<T, SRC, V>(g, x, x8, row, w.c, f);
        load_v<T, V>(gy + row * g.ys + g.yo + w.c, d);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          f[e] = xhat(f[e], mu[e], rs[e]);
          t[e] = affine(f[e], ga[e], be[e]);
        }
        slope_v<V>(g.act, t);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float du = d[e] * t[e];
          a[e] += du;
          b[e] = fmaf(du, f[e], b[e]);
        }
      }
    }
    join_rows<V>(k, sm, a);
    join_rows<V>(k, sm, b);
    if (w.rl == 0 && w.c < g.C) {
      float2* o = part + (w.n * k.chunks + w.chunk) * g.C + w.c;
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = make_float2(a[e], b[e]);
    }
  }
}

// sums[n][g] = (s1, s2) / count
template <typename T>
__global__ void __launch_bounds__(kNT)
group_sums_kernel(Norm g, Cut k, const float2* __restrict__ part, const T* __restrict__ gamma,
                  float2* __restrict__ sums) {
  __shared__ float sm[kNT / 32];
  for (int64_t i = blockIdx.x; i < g.N * g.G; i += gridDim.x) {
    const int64_t n = i / g.G;
    const int c0 = (int)(i - n * g.G) * g.D;
    const int64_t entries = (int64_t)k.chunks * g.D;
    float a = 0.f, b = 0.f;
    for (int64_t j = threadIdx.x; j < entries; j += kNT) {
      const int64_t ch = j / g.D;
      const int c = c0 + (int)(j - ch * g.D);
      const float2 p = part[(n * k.chunks + ch) * g.C + c];
      const float ga = gamma ? ld(gamma + c) : 1.f;
      a = fmaf(ga, p.x, a);
      b = fmaf(ga, p.y, b);
    }
    a = block_sum(a, sm);
    b = block_sum(b, sm);
    const float inv = 1.f / ((float)g.P * (float)g.D);
    if (threadIdx.x == 0) sums[i] = make_float2(a * inv, b * inv);
  }
}

// ggamma, gbeta from entries = N * chunks partial sums per channel: 32
// channels per block, 8 row lanes, a sum for every kRun entries of a lane
constexpr int kRun = 1024;
template <typename T>
__global__ void __launch_bounds__(kNT)
param_grad_kernel(int C, int64_t entries, const float2* __restrict__ part, T* __restrict__ ggamma,
                  T* __restrict__ gbeta) {
  __shared__ float2 sm[kNT];
  wait_for_previous();
  const int c = blockIdx.x * 32 + (threadIdx.x & 31);
  float a = 0.f, b = 0.f;
  if (c < C) {
    const float2* p = part + (threadIdx.x >> 5) * (int64_t)C + c;
    const int64_t step = (int64_t)(kNT / 32) * C;
    for (int64_t left = (entries - (threadIdx.x >> 5) + kNT / 32 - 1) / (kNT / 32); left > 0; left -= kRun) {
      const int n = (int)min(left, (int64_t)kRun);
      float u = 0.f, v = 0.f;
#pragma unroll 8
      for (int i = 0; i < n; ++i, p += step) {
        const float2 f = *p;
        u += f.x;
        v += f.y;
      }
      a += u;
      b += v;
    }
  }
  sm[threadIdx.x] = make_float2(a, b);
  __syncthreads();
  if (threadIdx.x < 32 && c < C) {
    for (int i = 1; i < kNT / 32; ++i) {
      a += sm[i * 32 + threadIdx.x].x;
      b += sm[i * 32 + threadIdx.x].y;
    }
    if (ggamma) ggamma[c] = from_f<T>(b);
    if (gbeta) gbeta[c] = from_f<T>(a);
  }
}

template <typename T, int SRC, int V>
__global__ void __launch_bounds__(kNT)
grad_apply_kernel(Norm g, Cut k, const T* __restrict__ x, Act8 x8, const T* __restrict__ gy,
                  const T* __restrict__ gamma, const T* __restrict__ beta, const float* __restrict__ mean,
                  const float* __restrict__ rstd, const float2* __restrict__ sums, T* __restrict__ gx) {
  for (int64_t i = blockIdx.x; i < k.units; i += gridDim.x) {
    const Unit w = unit_of<V>(g, k, k.units - 1 - i);
    if (w.c >= g.C) continue;
    float ga[V], be[V], mu[V], rs[V], s1[V], s2[V];
    load_affine<T, V>(g, w.c, gamma, beta, ga, be);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int64_t at = w.n * g.G + (w.c + e) / g.D;
      mu[e] = __ldg(mean + at);
      rs[e] = __ldg(rstd + at);
      const float2 s = sums[at];
      s1[e] = s.x;
      s2[e] = s.y;
    }
#pragma unroll 2
    for (int64_t r = w.r0 + w.rl; r < w.r1; r += k.rl) {
      const int64_t row = w.n * g.P + r;
      float f[V], d[V], t[V];
      load_src<T, SRC, V>(g, x, x8, row, w.c, f);
      load_v<T, V>(gy + row * g.ys + g.yo + w.c, d);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        f[e] = xhat(f[e], mu[e], rs[e]);
        t[e] = affine(f[e], ga[e], be[e]);
      }
      slope_v<V>(g.act, t);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float dv = d[e] * t[e] * ga[e];
        d[e] = (dv - fmaf(f[e], s2[e], s1[e])) * rs[e];
      }
      store_v<T, V>(gx + row * g.xs + g.xo + w.c, d);
    }
  }
}

unsigned grid_of(int64_t n) { return (unsigned)(n < (1 << 20) ? n : (1 << 20)); }

template <typename T, int V>
cudaError_t split_fwd(const Norm& g, const T* x, const T* gamma, const T* beta, T* y, float* mean, float* rstd,
                      float* ws, cudaStream_t s) {
  const Cut k = plan_cut(g, V);
  float2* stats = reinterpret_cast<float2*>(ws);
  float2* part = stats + g.N * g.G;
  moments_kernel<T, V><<<grid_of(k.units), kNT, 0, s>>>(g, k, x, part);
  group_moments_kernel<<<grid_of(g.N * g.G), kNT, 0, s>>>(g, k, part, stats, mean, rstd);
  apply_kernel<T, V><<<grid_of(k.units), kNT, 0, s>>>(g, k, x, gamma, beta, stats, y);
  return cudaGetLastError();
}

template <typename T, int SRC, int V>
cudaError_t split_bwd(const Norm& g, const T* x, const Act8& x8, const T* gy, const T* gamma, const T* beta,
                      const float* mean, const float* rstd, T* gx, T* ggamma, T* gbeta, float* ws,
                      cudaStream_t s) {
  const Cut k = plan_cut(g, V);
  float2* sums = reinterpret_cast<float2*>(ws);
  float2* part = sums + g.N * g.G;
  grad_sums_kernel<T, SRC, V><<<grid_of(k.units), kNT, 0, s>>>(g, k, x, x8, gy, gamma, beta, mean, rstd, part);
  if (ggamma || gbeta)
    param_grad_kernel<T><<<(g.C + 31) / 32, kNT, 0, s>>>(g.C, g.N * k.chunks, part, ggamma, gbeta);
  if (gx) {
    group_sums_kernel<T><<<grid_of(g.N * g.G), kNT, 0, s>>>(g, k, part, gamma, sums);
    grad_apply_kernel<T, SRC, V><<<grid_of(k.units), kNT, 0, s>>>(g, k, x, x8, gy, gamma, beta, mean, rstd, sums,
                                                                  gx);
  }
  return cudaGetLastError();
}

template <typename T, int V>
cudaError_t bwd_src(const Norm& g, const T* x, const Act8& x8, const T* gy, const T* gamma, const T* beta,
                    const float* mean, const float* rstd, T* gx, T* ggamma, T* gbeta, float* ws, cudaStream_t s) {
  if (x) return split_bwd<T, kSrcFull, V>(g, x, x8, gy, gamma, beta, mean, rstd, gx, ggamma, gbeta, ws, s);
  if (x8.src == kSrcI8)
    return split_bwd<T, kSrcI8, V>(g, x, x8, gy, gamma, beta, mean, rstd, gx, ggamma, gbeta, ws, s);
  return split_bwd<T, kSrcE4M3, V>(g, x, x8, gy, gamma, beta, mean, rstd, gx, ggamma, gbeta, ws, s);
}

template <typename T>
__global__ void zero_kernel(int C, T* a, T* b) {
  for (int c = blockIdx.x * blockDim.x + threadIdx.x; c < C; c += gridDim.x * blockDim.x) {
    if (a) a[c] = from_f<T>(0.f);
    if (b) b[c] = from_f<T>(0.f);
  }
}

}  // namespace

namespace {

int64_t lcm(int64_t a, int64_t b) {
  int64_t x = a, y = b;
  while (y) {
    const int64_t r = x % y;
    x = y;
    y = r;
  }
  return a / x * b;
}

// The layout of a pass: how a thread's channels lie, the slices and their
// rows; false: a slice wider than a block (the split kernels run). keep: the
// block of a checkpoint that the forward writes (0: none).
bool plan_slices(const Norm& g, int V, bool strided, int es, int keep, slab::Plan* out) {
  slab::Plan k{};
  k.V = V;
  k.strided = strided;
  if (keep && (strided || keep / V > 32)) return false;  // a block's lanes are one warp's
  int64_t base = strided ? g.D : lcm(g.D, V);
  if (keep && keep < g.C) base = lcm(base, keep);
  const int64_t line = 128 / es;
  int64_t S = base * ((line + base - 1) / base);
  if (S > g.C || keep >= g.C) S = g.C;  // a slice holds whole blocks of a checkpoint, or all channels
  k.S = (int)S;
  k.vpr = (int)((S + V - 1) / V);
  if (keep) k.vpr = (k.vpr + keep / V - 1) / (keep / V) * (keep / V);
  if (k.vpr > slab::kNT) return false;
  k.rl = slab::kNT / k.vpr;
  k.slices = (int)((g.C + S - 1) / S);
  k.groups = (int)(S / g.D);
  k.d_vpr = FastDiv((uint32_t)k.vpr);
  k.d_slices = FastDiv((uint32_t)k.slices);
  k.d_D = FastDiv((uint32_t)g.D);
  k.total = (float)g.P * (float)g.D;
  k.inv_total = 1.f / k.total;
  k.inv_D = 1.f / (float)g.D;
  *out = k;
  return true;
}

// Bytes of shared memory that a vector of a row takes. x_bytes: of an element
// of the backward's input (0: forward; 1: codes, with their scales).
int64_t vector_bytes(const slab::Plan& k, int es, int x_bytes) {
  return k.V * (es + x_bytes) + (x_bytes == 1 ? (k.strided ? 4 * k.V : 4) : 0);
}

constexpr int kFewRows = 8;

// Clusters of up to eight blocks that hold a slab: the size whose blocks, in
// whole waves of as many as an SM holds at a time, issue the fewest
// instructions. A block costs about 900 per warp and 28 per element and row
// lane (20 forward); an SM with one, two and three blocks issues at about
// 0.25, 0.42 and 0.54 of its rate (ncu).
bool plan_cluster(const Norm& g, int es, int x_bytes, slab::Plan* k) {
  const int64_t units = g.N * k->slices, row = k->vpr * vector_bytes(*k, es, x_bytes);
  const int pass = x_bytes ? 1 : 0, scratch = slab::scratch_bytes(*k, pass), most = pass && k->V == 8 ? 2 : 3;
  double best = -1;
  for (int parts = 1; parts <= 8; ++parts) {
    const int64_t rows = (g.P + parts - 1) / parts;
    if (parts > 1 && (rows < k->rl || rows * (parts - 1) >= g.P)) continue;  // a block without rows
    const int64_t data = (rows * row + 15) / 16 * 16;
    if (data + scratch > slab::kMostSmem || units * parts >= (int64_t(1) << 31)) continue;
    int64_t blocks = 226 * 1024 / (data + scratch + 1024);
    if (blocks > most) blocks = most;
    const int64_t here = units * parts, wave = 152 * blocks, waves = (here + wave - 1) / wave;
    int64_t busy = (here + 151) / 152;  // blocks that the fullest SM holds at a time
    if (busy > blocks) busy = blocks;
    const double rate = busy == 1 ? 0.25 : busy == 2 ? 0.42 : 0.54;
    const double lane_rows = (double)((rows + k->rl - 1) / k->rl);
    const double cost = (double)waves * busy * (900 + (pass ? 28 : 20) * k->V * lane_rows) / rate;
    if (best >= 0 && cost >= best) continue;
    best = cost;
    k->parts = parts;
    k->rows = (int)rows;
    k->data_bytes = (int)data;
  }
  if (best < 0) return false;
  k->d_parts = FastDiv((uint32_t)k->parts);
  return units * k->parts >= 152 || k->rows <= kFewRows * k->rl;  // too few blocks for so many rows: stream
}

constexpr int kStreamBlocks = 3;

// Chunks of pixels for the stream kernels: one wave of blocks (at
// 2x256x256x64 fp32: 29 us at six blocks per SM, 27 at four, 23 at three), at
// least four rows for a row lane and at most kChain.
bool plan_stream(const Norm& g, int es, int x_bytes, slab::Plan* k) {
  const int64_t units = g.N * k->slices;
  int64_t parts = (152 * kStreamBlocks + units - 1) / units;
  const int64_t chains = (g.P + kChain * k->rl - 1) / (kChain * k->rl), most = (g.P + 4 * k->rl - 1) / (4 * k->rl);
  if (parts < chains) parts = chains;
  if (parts > most) parts = most;
  if (parts > slab::kMaxParts) parts = slab::kMaxParts;
  const int64_t rows = (g.P + parts - 1) / parts;
  if (rows >= (int64_t(1) << 31)) return false;
  k->rows = (int)rows;
  k->parts = (int)((g.P + rows - 1) / rows);
  k->d_parts = FastDiv((uint32_t)k->parts);
  k->data_bytes = (int)(2 * slab::kBatch * slab::kNT * vector_bytes(*k, es, x_bytes));
  return units * k->parts < (int64_t(1) << 31) &&
         k->data_bytes + slab::scratch_bytes(*k, x_bytes ? 1 : 0) <= slab::kMostSmem;
}

enum Family { kSlabs, kStream, kSplit };

Family plan_family(const Norm& g, int V, bool strided, int es, int keep, int x_bytes, slab::Plan* k) {
  if (!plan_slices(g, V, strided, es, keep, k)) return kSplit;
  if (plan_cluster(g, es, x_bytes, k)) return kSlabs;
  return plan_stream(g, es, x_bytes, k) ? kStream : kSplit;
}

// How a thread's channels lie: the widest access that distances, offsets and
// pointers allow (16 bytes; 8 for 16-bit types), or four channels apart.
void layout_of(const Norm& g, int es, int widest, const void* a, const void* b, const void* c, const void* codes, int* V,
               bool* strided) {
  for (int bytes : {16, 8}) {
    *V = bytes / es;
    if (*V < 4 || *V > widest) continue;
    auto fits = [&](const void* p) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; };
    if (g.C % *V == 0 && g.xs % *V == 0 && g.xo % *V == 0 && g.ys % *V == 0 && g.yo % *V == 0 && fits(a) && fits(b) &&
        fits(c) && reinterpret_cast<uintptr_t>(codes) % *V == 0) {
      *strided = false;
      return;
    }
  }
  *V = 4;
  *strided = true;
}

int elem_size(int dtype) { return dtype == DWCONV_F32 ? 4 : 2; }

}  // namespace

const char* plan_name(const Norm& g, int pass) {
  const int es = elem_size(g.dtype);
  int V;
  bool strided;
  slab::Plan k;
  layout_of(g, es, pass ? 4 : 8, nullptr, nullptr, nullptr, nullptr, &V, &strided);
  const Family f = plan_family(g, V, strided, es, 0, pass ? es : 0, &k);
  return f == kSlabs ? "slab" : f == kStream ? "stream" : "split";
}

// Sums per part and group and, in the backward, per part and channel, for the
// family and layout with the most parts that a call's pointers may lead to.
size_t workspace_bytes(const Norm& g, int pass) {
  if (g.N == 0) return 0;
  const int es = elem_size(g.dtype);
  int64_t parts = 1;
  bool split_too = false;
  for (int V : {8, 4, 1}) {  // 1: channels apart
    slab::Plan k;
    if (V * es > 16) continue;
    if (plan_slices(g, V == 1 ? 4 : V, V == 1, es, 0, &k) && plan_stream(g, es, pass ? es : 0, &k)) {
      if (k.parts > parts) parts = k.parts;
    } else {
      split_too = true;
    }
    // a checkpoint's blocks widen the slices
    for (int keep : {32, 64, 128})
      if (V > 1 && plan_slices(g, V, false, es, keep, &k) && plan_stream(g, es, 0, &k) && k.parts > parts) parts = k.parts;
  }
  size_t pairs = (size_t)g.N * (size_t)parts * ((size_t)g.G + (pass ? (size_t)g.C : 0));
  const int64_t a = plan_cut(g, 1).chunks, b = plan_cut(g, 16 / es).chunks;
  const size_t split = (size_t)(g.N * g.G) + (size_t)g.N * (size_t)(a > b ? a : b) * (size_t)g.C;
  if (split_too && split > pairs) pairs = split;
  return (pairs * sizeof(float2) + 255) & ~size_t(255);
}

namespace {

template <typename T>
cudaError_t fwd_any(const Norm& g, const T* x, const T* gamma, const T* beta, T* y, float* mean, float* rstd, float* ws,
                    const Act8& x8, cudaStream_t s) {
  const int es = sizeof(T), block = x8.codes ? 1 << x8.shift : 0;
  int V;
  bool strided;
  layout_of(g, es, 8, x, y, nullptr, x8.codes, &V, &strided);
  const slab::Sums sums{reinterpret_cast<float2*>(ws), nullptr};
  slab::Plan k;
  Family f = block ? plan_family(g, V, strided, es, block, 0, &k) : kSplit;
  if (f != kSplit) return slab::run_fwd<T>(g, k, f == kSlabs, x, gamma, beta, y, mean, rstd, x8, sums, s);
  cudaError_t e;
  f = plan_family(g, V, strided, es, 0, 0, &k);
  if (f != kSplit) {
    e = slab::run_fwd<T>(g, k, f == kSlabs, x, gamma, beta, y, mean, rstd, Act8{}, sums, s);
  } else {
    constexpr int VV = Vec<T>::n;
    e = V == VV && !strided ? split_fwd<T, VV>(g, x, gamma, beta, y, mean, rstd, ws, s)
                            : split_fwd<T, 1>(g, x, gamma, beta, y, mean, rstd, ws, s);
  }
  if (e == cudaSuccess && block) e = act8_encode(g.N * g.P, g.C, g.xs, g.dtype, x + g.xo, x8, s);
  return e;
}

template <typename T>
cudaError_t bwd_any(const Norm& g, const T* x, const Act8& x8, const T* gy, const T* gamma, const T* beta,
                    const float* mean, const float* rstd, T* gx, T* ggamma, T* gbeta, float* ws, cudaStream_t s) {
  if (g.N == 0) {
    if (!ggamma && !gbeta) return cudaSuccess;
    zero_kernel<T><<<(unsigned)div_up(g.C, 256), 256, 0, s>>>(g.C, ggamma, gbeta);
    return cudaGetLastError();
  }
  const int es = sizeof(T);
  int V;
  bool strided;
  // eight channels of x and gy in full take 125 registers and two blocks per SM, four 80 and three: 45 against 39 us at
  // 64x28x28x256 bf16; from codes eight are faster, 125 against 137 us for the step at 64x56x56x128
  layout_of(g, es, x ? 4 : 8, x, gy, gx, x8.codes, &V, &strided);
  slab::Plan k;
  const Family f = plan_family(g, V, strided, es, 0, x ? es : 1, &k);
  if (f != kSplit) {
    const int64_t parts = f == kSlabs ? 1 : k.parts;
    slab::Sums sums;
    sums.channels = reinterpret_cast<float2*>(ws);
    sums.groups = sums.channels + g.N * parts * g.C;
    const cudaError_t e = slab::run_bwd<T>(g, k, f == kSlabs, x, x8, gy, gamma, beta, mean, rstd, gx, sums, s);
    if (e != cudaSuccess || (!ggamma && !gbeta)) return e;
    return launch_dependent(param_grad_kernel<T>, dim3((g.C + 31) / 32), dim3(kNT), 0, s, g.C, (int64_t)(g.N * parts),
                            (const float2*)sums.channels, ggamma, gbeta);
  }
  constexpr int VV = Vec<T>::n;
  return V == VV && !strided ? bwd_src<T, VV>(g, x, x8, gy, gamma, beta, mean, rstd, gx, ggamma, gbeta, ws, s)
                             : bwd_src<T, 1>(g, x, x8, gy, gamma, beta, mean, rstd, gx, ggamma, gbeta, ws, s);
}

}  // namespace

cudaError_t fwd(const Norm& g, const void* x, const void* gamma, const void* beta, void* y, float* mean,
                float* rstd, float* ws, const Act8& x8, cudaStream_t s) {
  cudaError_t e = cudaErrorInvalidValue;
  DWCONV_DISPATCH_DTYPE(g.dtype, T, e = fwd_any<T>(g, (const T*)x, (const T*)gamma, (const T*)beta, (T*)y, mean, rstd,
                                                   ws, x8, s));
  return e;
}

cudaError_t bwd(const Norm& g, const void* x, const Act8& x8, const void* gy, const void* gamma,
                const void* beta, const float* mean, const float* rstd, void* gx, void* ggamma, void* gbeta,
                float* ws, cudaStream_t s) {
  cudaError_t e = cudaErrorInvalidValue;
  DWCONV_DISPATCH_DTYPE(g.dtype, T, e = bwd_any<T>(g, (const T*)x, x8, (const T*)gy, (const T*)gamma, (const T*)beta,
                                                   mean, rstd, (T*)gx, (T*)ggamma, (T*)gbeta, ws, s));
  return e;
}

}  // namespace norm
}  // namespace dwconv
