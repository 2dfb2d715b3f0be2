// Channels-last group norm, forward and backward: the slab kernels, which
// read their inputs once.
//
// A unit of work is a slab: one sample's pixels times a slice of channels
// that holds whole groups, at least one 128-byte line wide where the channels
// allow it. A cluster of thread blocks owns a slab, each block a share of its
// pixels: it reads them once, 16 bytes per thread and access, takes the sums
// on the way and leaves the data as read in shared memory; the blocks join
// their sums through the cluster's distributed shared memory; then each
// writes its outputs from its own shared memory. Bytes moved are the floor's:
// inputs once, outputs once. The forward also writes the 8-bit checkpoint of
// x from the registers that hold it (a block of channels is a few
// neighbouring lanes).
//
// Slabs that no cluster of eight blocks can hold, and slices wider than a
// block, are left to the split kernels (norm.cu).
//
// The variance is joined as in norm.cu: a thread sums x - s and (x - s)^2
// about its own first value s of a channel, the squares are moved to the
// block's mean of the group, and the blocks' (count, mean, squares) are
// joined by the parallel form. Every order is fixed.
#pragma once

#include <cooperative_groups.h>

#include "norm.cuh"
#include "norm_slab.h"

namespace dwconv {
namespace norm {
namespace slab {

namespace cg = cooperative_groups;

// V elements as they are stored: 16 bytes, 4 bytes or one element
template <int BYTES> struct Word;
template <> struct Word<16> { typedef uint4 type; };
template <> struct Word<8> { typedef uint2 type; };
template <> struct Word<4> { typedef uint32_t type; };
template <> struct Word<2> { typedef uint16_t type; };
template <> struct Word<1> { typedef uint8_t type; };

template <typename T, int V>
struct Vecs {
  typedef typename Word<V * (int)sizeof(T)>::type word;
  static __device__ __forceinline__ void unpack(word w, float* f) {
    if constexpr (V * sizeof(T) == 16) {
      unpack16<T>(w, f);
    } else {
      const T* p = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = to_f<T>(p[e]);
    }
  }
  static __device__ __forceinline__ word pack(const float* f) {
    if constexpr (V * sizeof(T) == 16) {
      return pack16<T>(f);
    } else {
      word w;
      T* p = reinterpret_cast<T*>(&w);
#pragma unroll
      for (int e = 0; e < V; ++e) p[e] = from_f<T>(f[e]);
      return w;
    }
  }
};

// codes of V values
template <int SRC, int V>
__device__ __forceinline__ void unpack_codes(typename Word<V>::type w, float s, float* f) {
  if constexpr (V == 8) {
    codes4<SRC>(w.x, f);
    codes4<SRC>(w.y, f + 4);
  } else if constexpr (V == 4) {
    codes4<SRC>(w, f);
  } else {
    float o[4];
    codes4<SRC>((uint32_t)w, o);
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = o[e];
  }
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = __fmul_rn(f[e], s);
}
template <int SRC, int V>
__device__ __forceinline__ typename Word<V>::type pack_codes(const float* f, float inv) {
  if constexpr (V == 8) {
    return make_uint2(encode4<SRC>(f[0], f[1], f[2], f[3], inv), encode4<SRC>(f[4], f[5], f[6], f[7], inv));
  } else if constexpr (V == 4) {
    return encode4<SRC>(f[0], f[1], f[2], f[3], inv);
  } else if constexpr (V == 2) {
    return (uint16_t)encode4<SRC>(f[0], f[1], 0.f, 0.f, inv);
  } else {
    return encode1<SRC>(f[0], inv);
  }
}

// Sums v over the block's row lanes, in lane order, into chan[channel of the
// slice]; red holds kNT * V floats.
template <int V>
__device__ __forceinline__ void join_rows(const Plan& k, const float* v, float* red, float* chan) {
  const int n = k.vpr * V;  // channels, idle ones included
  const bool in = (int)threadIdx.x < k.rl * k.vpr;
  __syncthreads();
  if (in) {
#pragma unroll
    for (int e = 0; e < V; ++e) red[e * kNT + threadIdx.x] = v[e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kNT) {
    const int e = i / k.vpr, vl = i - e * k.vpr;
    float a = 0.f;
#pragma unroll 8
    for (int r = 0; r < k.rl; ++r) a += red[e * kNT + r * k.vpr + vl];
    chan[vl * V + e] = a;
  }
  __syncthreads();
}

// sum over the D channels of a group, one warp, in a fixed order
template <typename F>
__device__ __forceinline__ float warp_sum(int D, F value) {
  float a = 0.f;
  for (int c = threadIdx.x & 31; c < D; c += 32) a += value(c);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  return a;
}

// shared memory after the shares: red, then per channel and per group tables
template <int V>
__device__ __forceinline__ float* scratch(unsigned char* sm, const Plan& k) {
  return reinterpret_cast<float*>(sm + k.data_bytes);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// group of the slice that each of a vector's channels belongs to
template <int V>
__device__ __forceinline__ void groups_of(int D, int first, int* gi) {
  int q = first / D, r = first - q * D;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    gi[e] = q;
    if (++r == D) {
      r = 0;
      ++q;
    }
  }
}

struct Place {
  int64_t n, row0;   // sample, first row of the share in the tensor
  int rows;          // of the share (0: none)
  int c0, S;         // first channel and channels of the slice
  int c, vl, r;      // this thread's first channel, vector and row lane
  bool on;           // has channels
};

template <int V>
__device__ __forceinline__ Place place_of(const Norm& g, const Plan& k) {
  Place p;
  const uint32_t unit = blockIdx.x / k.cl, rank = blockIdx.x - unit * k.cl;
  p.n = unit / k.slices;
  const int slice = (int)(unit - (uint32_t)p.n * k.slices);
  p.c0 = slice * k.S;
  p.S = min(k.S, g.C - p.c0);
  const int64_t r0 = (int64_t)rank * k.rows;
  p.rows = (int)(r0 < g.P ? (g.P - r0 < k.rows ? g.P - r0 : k.rows) : 0);
  p.row0 = p.n * g.P + r0;
  p.r = threadIdx.x / k.vpr;
  p.vl = threadIdx.x - p.r * k.vpr;
  p.c = p.c0 + p.vl * V;
  p.on = p.r < k.rl && p.vl * V < p.S;
  return p;
}

template <typename T, int V, int KEEP>
__global__ void __launch_bounds__(kNT)
fwd_kernel(Norm g, Plan k, const T* __restrict__ x, const T* __restrict__ gamma, const T* __restrict__ beta,
           T* __restrict__ y, float* __restrict__ mean_out, float* __restrict__ rstd_out, Act8 x8) {
  typedef typename Vecs<T, V>::word word;
  extern __shared__ __align__(16) unsigned char sm[];
  cg::cluster_group cluster = cg::this_cluster();
  const Place p = place_of<V>(g, k);
  word* const data = reinterpret_cast<word*>(sm);
  float* const red = scratch<V>(sm, k);
  float* const chan = red + kNT * V;
  float2* const part = reinterpret_cast<float2*>(chan + (k.vpr * V + 1) / 2 * 2);  // (mean, squares) of the block's groups
  float2* const stat = part + k.groups;                             // (mean, rstd) of the slab's

  // read, sum, keep
  float s[V], d[V], q[V];
#pragma unroll
  for (int e = 0; e < V; ++e) s[e] = d[e] = q[e] = 0.f;
  int gi[V];
  groups_of<V>(g.D, min(p.vl * V, p.S - 1), gi);
  const T* xp = x + p.row0 * g.xs + g.xo + p.c;
  constexpr int kAhead = V == 1 ? 8 : 4;  // rows in flight
  for (int r0 = 0; r0 < p.rows; r0 += kAhead * k.rl) {
    word w[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int r = r0 + a * k.rl + p.r;
      w[a] = word{};
      if (p.on && r < p.rows) w[a] = *reinterpret_cast<const word*>(xp + (int64_t)r * g.xs);
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int r = r0 + a * k.rl + p.r;
      const bool in = p.on && r < p.rows;
      float f[V];
      Vecs<T, V>::unpack(w[a], f);
      if (in) {
        data[r * k.vpr + p.vl] = w[a];
        if (a == 0 && r0 == 0) {
#pragma unroll
          for (int e = 0; e < V; ++e) s[e] = f[e];
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float t = f[e] - s[e];
          d[e] += t;
          q[e] = fmaf(t, t, q[e]);
        }
      }
      if (KEEP != kSrcFull) {  // lanes of a block of channels are neighbours; those without data bring zeros
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < V; ++e) m = max(m, abs_bits(f[e]));
        for (int o = (1 << x8.shift) / V >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (in) {
          float inv;
          const float sc = scale_of<KEEP>(m, &inv);
          typedef typename Word<V>::type codes;
          *reinterpret_cast<codes*>(x8.codes + (p.row0 + r) * g.C + p.c) = pack_codes<KEEP, V>(f, inv);
          if ((p.c & ((1 << x8.shift) - 1)) == 0) x8.scales[(p.row0 + r) * x8.nblk + (p.c >> x8.shift)] = sc;
        }
      }
    }
  }

  // the block's mean and squares of each group
  const int mine = p.on && p.r < p.rows ? (p.rows - p.r + k.rl - 1) / k.rl : 0;
  const float cnt = (float)mine, icnt = mine > 0 ? 1.f / cnt : 0.f;
  const int warp = threadIdx.x >> 5, groups = p.S / g.D;
  {
    float v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = fmaf(cnt, s[e], d[e]);
    join_rows<V>(k, v, red, chan);
    for (int i = warp; i < groups; i += kNT / 32) {
      const float a = warp_sum(g.D, [&](int c) { return chan[i * g.D + c]; });
      if ((threadIdx.x & 31) == 0) part[i].x = p.rows > 0 ? a / ((float)p.rows * (float)g.D) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float m = fmaf(d[e], icnt, s[e]);
      const float own = q[e] - d[e] * d[e] * icnt;
      const float t = p.on ? m - part[gi[e]].x : 0.f;
      v[e] = mine > 0 ? (own < 0.f ? 0.f : own) + cnt * t * t : 0.f;  // NaN stays
    }
    join_rows<V>(k, v, red, chan);
    for (int i = warp; i < groups; i += kNT / 32) {
      const float a = warp_sum(g.D, [&](int c) { return chan[i * g.D + c]; });
      if ((threadIdx.x & 31) == 0) part[i].y = a;
    }
  }
  // the slab's
  cluster_arrive();
  cluster_wait();
  for (int i = threadIdx.x; i < groups; i += kNT) {
    const float total = (float)g.P * (float)g.D;
    float a = 0.f;
    for (int b = 0; b < k.cl; ++b) {
      const int64_t r0 = (int64_t)b * k.rows;
      const float n = (float)(r0 < g.P ? min((int64_t)k.rows, g.P - r0) : 0) * (float)g.D;
      a = fmaf(n, cluster.map_shared_rank(part, b)[i].x, a);
    }
    const float mean = a / total;
    float sq = 0.f;
    for (int b = 0; b < k.cl; ++b) {
      const int64_t r0 = (int64_t)b * k.rows;
      const float n = (float)(r0 < g.P ? min((int64_t)k.rows, g.P - r0) : 0) * (float)g.D;
      const float2 o = cluster.map_shared_rank(part, b)[i];
      const float t = o.x - mean;
      sq += n > 0.f ? fmaf(n * t, t, o.y) : 0.f;
    }
    const float rstd = 1.f / sqrtf(sq / total + g.eps);
    stat[i] = make_float2(mean, rstd);
    if (cluster.block_rank() == 0) {
      const int64_t at = p.n * g.G + p.c0 / g.D + i;
      if (mean_out) mean_out[at] = mean;
      if (rstd_out) rstd_out[at] = rstd;
    }
  }
  __syncthreads();
  if (k.cl > 1) cluster_arrive();  // this block has read the others' sums

  // write
  if (p.on) {
    float ga[V], be[V], mu[V], rs[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      ga[e] = gamma ? ld(gamma + p.c + e) : 1.f;
      be[e] = beta ? ld(beta + p.c + e) : 0.f;
      const float2 st = stat[gi[e]];
      mu[e] = st.x;
      rs[e] = st.y;
    }
    T* yp = y + p.row0 * g.ys + g.yo + p.c;
#pragma unroll 2
    for (int r = p.r; r < p.rows; r += k.rl) {
      float f[V];
      Vecs<T, V>::unpack(data[r * k.vpr + p.vl], f);
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = affine(xhat(f[e], mu[e], rs[e]), ga[e], be[e]);
      act_v<V>(g.act, f);
      *reinterpret_cast<word*>(yp + (int64_t)r * g.ys) = Vecs<T, V>::pack(f);
    }
  }
  if (k.cl > 1) cluster_wait();  // no block leaves while another reads its sums
}

template <typename T, int V, int SRC>
__global__ void __launch_bounds__(kNT)
bwd_kernel(Norm g, Plan k, const T* __restrict__ x, Act8 x8, const T* __restrict__ gy, const T* __restrict__ gamma,
           const T* __restrict__ beta, const float* __restrict__ mean, const float* __restrict__ rstd,
           T* __restrict__ gx, float2* __restrict__ sums) {
  typedef typename Vecs<T, V>::word word;
  typedef typename Word<SRC == kSrcFull ? V * (int)sizeof(T) : V>::type xword;
  extern __shared__ __align__(16) unsigned char sm[];
  cg::cluster_group cluster = cg::this_cluster();
  const Place p = place_of<V>(g, k);
  word* const gdata = reinterpret_cast<word*>(sm);
  xword* const xdata = reinterpret_cast<xword*>(sm + (size_t)k.rows * k.vpr * sizeof(word));
  float* const red = scratch<V>(sm, k);
  float* const chan = red + kNT * V;                                            // sum du, then sum du * xh
  float2* const part = reinterpret_cast<float2*>(chan + 2 * k.vpr * V);         // (s1, s2) of the block's groups
  float2* const stat = part + k.groups;                                         // of the slab's, over the count

  int gi[V];
  groups_of<V>(g.D, min(p.vl * V, p.S - 1), gi);
  float ga[V], be[V], mu[V], rs[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    ga[e] = be[e] = mu[e] = rs[e] = 0.f;
    if (p.on) {
      ga[e] = gamma ? ld(gamma + p.c + e) : 1.f;
      be[e] = beta ? ld(beta + p.c + e) : 0.f;
      const int64_t at = p.n * g.G + p.c0 / g.D + gi[e];
      mu[e] = __ldg(mean + at);
      rs[e] = __ldg(rstd + at);
    }
  }
  const T* gp = gy + p.row0 * g.ys + g.yo + p.c;
  auto load_x = [&](int r) {
    if constexpr (SRC == kSrcFull) {
      return *reinterpret_cast<const xword*>(x + (p.row0 + r) * g.xs + g.xo + p.c);
    } else {
      return *reinterpret_cast<const xword*>(x8.codes + (p.row0 + r) * g.C + p.c);
    }
  };
  auto scale_at = [&](int r) {
    return SRC == kSrcFull ? 0.f : __ldg(x8.scales + (p.row0 + r) * x8.nblk + (p.c >> x8.shift));
  };
  // xh and du of one vector, from what was stored
  auto eval = [&](word gw, xword xw, float sc, float* xh, float* du) {
    float t[V];
    if constexpr (SRC == kSrcFull) {
      Vecs<T, V>::unpack(xw, xh);
    } else {
      unpack_codes<SRC, V>(xw, sc, xh);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      xh[e] = xhat(xh[e], mu[e], rs[e]);
      t[e] = affine(xh[e], ga[e], be[e]);
    }
    slope_v<V>(g.act, t);
    Vecs<T, V>::unpack(gw, du);
#pragma unroll
    for (int e = 0; e < V; ++e) du[e] *= t[e];
  };

  // read, sum, keep
  float a[V], b[V];
#pragma unroll
  for (int e = 0; e < V; ++e) a[e] = b[e] = 0.f;
  if (p.on) {
    constexpr int kAhead = V == 1 ? 4 : 2;
    for (int r0 = p.r; r0 < p.rows; r0 += kAhead * k.rl) {
      word gw[kAhead];
      xword xw[kAhead];
      float sc[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int r = r0 + i * k.rl;
        gw[i] = word{};
        xw[i] = xword{};
        sc[i] = 0.f;
        if (r < p.rows) {
          gw[i] = *reinterpret_cast<const word*>(gp + (int64_t)r * g.ys);
          xw[i] = load_x(r);
          sc[i] = scale_at(r);
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int r = r0 + i * k.rl;
        if (r >= p.rows) break;
        gdata[r * k.vpr + p.vl] = gw[i];
        xdata[r * k.vpr + p.vl] = xw[i];
        float xh[V], du[V];
        eval(gw[i], xw[i], sc[i], xh, du);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          a[e] += du[e];
          b[e] = fmaf(du[e], xh[e], b[e]);
        }
      }
    }
  }
  float* const chan2 = chan + k.vpr * V;
  join_rows<V>(k, a, red, chan);
  join_rows<V>(k, b, red, chan2);
  const int warp = threadIdx.x >> 5, groups = p.S / g.D;
  for (int i = warp; i < groups; i += kNT / 32) {
    auto ga_of = [&](int c) { return gamma ? ld(gamma + p.c0 + i * g.D + c) : 1.f; };
    const float s1 = warp_sum(g.D, [&](int c) { return ga_of(c) * chan[i * g.D + c]; });
    const float s2 = warp_sum(g.D, [&](int c) { return ga_of(c) * chan2[i * g.D + c]; });
    if ((threadIdx.x & 31) == 0) part[i] = make_float2(s1, s2);
  }
  cluster_arrive();
  cluster_wait();
  const float inv = 1.f / ((float)g.P * (float)g.D);
  for (int i = threadIdx.x; i < groups; i += kNT) {
    float s1 = 0.f, s2 = 0.f;
    for (int j = 0; j < k.cl; ++j) {
      const float2 o = cluster.map_shared_rank(part, j)[i];
      s1 += o.x;
      s2 += o.y;
    }
    stat[i] = make_float2(s1 * inv, s2 * inv);
  }
  // the slab's sums per channel, each block its share of the channels
  const int share = (p.S + k.cl - 1) / k.cl, lo = (int)cluster.block_rank() * share;
  for (int c = lo + threadIdx.x; c < min(lo + share, p.S); c += kNT) {
    float s1 = 0.f, s2 = 0.f;
    for (int j = 0; j < k.cl; ++j) {
      s1 += cluster.map_shared_rank(chan, j)[c];
      s2 += cluster.map_shared_rank(chan2, j)[c];
    }
    sums[p.n * g.C + p.c0 + c] = make_float2(s1, s2);
  }
  __syncthreads();
  if (k.cl > 1) cluster_arrive();

  // write
  if (gx && p.on) {
    float s1[V], s2[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float2 st = stat[gi[e]];
      s1[e] = st.x;
      s2[e] = st.y;
    }
    T* op = gx + p.row0 * g.xs + g.xo + p.c;
    for (int r = p.r; r < p.rows; r += k.rl) {
      float xh[V], du[V];
      eval(gdata[r * k.vpr + p.vl], xdata[r * k.vpr + p.vl], scale_at(r), xh, du);
#pragma unroll
      for (int e = 0; e < V; ++e) du[e] = (du[e] * ga[e] - fmaf(xh[e], s2[e], s1[e])) * rs[e];
      *reinterpret_cast<word*>(op + (int64_t)r * g.xs) = Vecs<T, V>::pack(du);
    }
  }
  if (k.cl > 1) cluster_wait();
}

// ---- launches --------------------------------------------------------------

template <typename... P, typename... A>
cudaError_t launch(void (*kern)(P...), const Norm& g, const Plan& k, int V, int pass, cudaStream_t s, A... args) {
  const int smem = k.data_bytes + scratch_bytes(k, V, pass);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)k.cl;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(g.N * k.slices * k.cl));
  cfg.blockDim = dim3(kNT);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// V of a type: 16 bytes, 4 bytes, one element
#define DW_SLAB_V(X)                                       \
  if (V * (int)sizeof(T) == 16) { X(16 / (int)sizeof(T)) } \
  if constexpr (sizeof(T) == 2) {                          \
    if (V == 2) { X(2) }                                   \
  }                                                        \
  if (V == 1) { X(1) }

template <typename T>
cudaError_t run_fwd(const Norm& g, const Plan& k, int V, const T* x, const T* gamma, const T* beta, T* y, float* mean,
                    float* rstd, const Act8& x8, cudaStream_t s) {
  const int keep = x8.codes ? x8.src : kSrcFull;
#define Y(VV, KEEP) \
  if (keep == KEEP) return launch(fwd_kernel<T, VV, KEEP>, g, k, V, 0, s, g, k, x, gamma, beta, y, mean, rstd, x8);
#define X(VV) Y(VV, kSrcFull) Y(VV, kSrcI8) Y(VV, kSrcE4M3)
  DW_SLAB_V(X)
#undef X
#undef Y
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t run_bwd(const Norm& g, const Plan& k, int V, const T* x, const Act8& x8, const T* gy, const T* gamma,
                    const T* beta, const float* mean, const float* rstd, T* gx, float2* sums, cudaStream_t s) {
  const int src = x ? kSrcFull : x8.src;
#define Y(VV, SRC) \
  if (src == SRC)  \
    return launch(bwd_kernel<T, VV, SRC>, g, k, V, 1, s, g, k, x, x8, gy, gamma, beta, mean, rstd, gx, sums);
#define X(VV) Y(VV, kSrcFull) Y(VV, kSrcI8) Y(VV, kSrcE4M3)
  DW_SLAB_V(X)
#undef X
#undef Y
  return cudaErrorInvalidValue;
}

}  // namespace slab
}  // namespace norm
}  // namespace dwconv
