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
// The variance is not taken from sums of squares of x: a block sums x - s and
// (x - s)^2 about the values s of its first pixel, one per channel, turns
// them into a mean and squares about that mean, and joins channels and blocks
// by the parallel form of the two (see norm.cu). Every order is fixed.
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

// V elements as pairs (an odd V's last pair has 0 in its second lane)
template <typename T, int V>
struct Vecs {
  typedef typename Word<V * (int)sizeof(T)>::type word;
  static constexpr int NP = (V + 1) / 2;
  static __device__ __forceinline__ void unpack(word w, f32x2* f) {
    if constexpr (V * sizeof(T) == 16) {
      unpack16_pairs<T>(w, f);
    } else {
      const T* p = reinterpret_cast<const T*>(&w);
      f[0] = pack_f32x2(to_f<T>(p[0]), V > 1 ? to_f<T>(p[V - 1]) : 0.f);
    }
  }
  static __device__ __forceinline__ word pack(const f32x2* f) {
    float v[2 * NP];
#pragma unroll
    for (int e = 0; e < NP; ++e) unpack_f32x2(f[e], v[2 * e], v[2 * e + 1]);
    if constexpr (V * sizeof(T) == 16) {
      return pack16<T>(v);
    } else {
      word w;
      T* p = reinterpret_cast<T*>(&w);
#pragma unroll
      for (int e = 0; e < V; ++e) p[e] = from_f<T>(v[e]);
      return w;
    }
  }
};

// codes of V values
template <int SRC, int V>
__device__ __forceinline__ void unpack_codes(typename Word<V>::type w, float s, f32x2* f) {
  if constexpr (V == 8) {
    decode4<SRC>(w.x, s, f);
    decode4<SRC>(w.y, s, f + 2);
  } else if constexpr (V == 4) {
    decode4<SRC>(w, s, f);
  } else {
    f32x2 o[2];
    decode4<SRC>((uint32_t)w, s, o);
    f[0] = o[0];
  }
}
template <int SRC, int V>
__device__ __forceinline__ typename Word<V>::type pack_codes(const f32x2* f, float inv) {
  if constexpr (V == 8) {
    return make_uint2(encode4<SRC>(f[0], f[1], inv), encode4<SRC>(f[2], f[3], inv));
  } else if constexpr (V == 4) {
    return encode4<SRC>(f[0], f[1], inv);
  } else {
    return (typename Word<V>::type)encode4<SRC>(f[0], 0, inv);
  }
}

// The largest pattern without sign of a vector's values and its neighbours'
// of a block of channels (`lanes` of them), as that of an fp32 value.
// Patterns of 16-bit types are compared two at a time.
template <typename T, int V>
__device__ __forceinline__ uint32_t block_max(typename Vecs<T, V>::word w, int lanes) {
  if constexpr (sizeof(T) == 4) {
    uint32_t m = 0;
    const uint32_t* u = reinterpret_cast<const uint32_t*>(&w);
#pragma unroll
    for (int e = 0; e < V; ++e) m = max(m, u[e] & 0x7fffffffu);
    for (int o = lanes >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
  } else {
    uint32_t m;
    if constexpr (V == 8) {
      m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
    } else {
      m = (uint32_t)w & 0x7fff7fffu;
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    const unsigned short h = (unsigned short)max(m & 0xffffu, m >> 16);
    return __float_as_uint(to_f<T>(*reinterpret_cast<const T*>(&h)));
  }
}

// Sums two vectors over the block's row lanes, in lane order. Afterwards
// tot[vl * 4 NP + e] is the sum of u's element e of vector vl of the slice
// and tot[vl * 4 NP + 2 NP + e] that of v's. red holds kNT * 4 NP floats.
template <int NP>
__device__ __forceinline__ void join_rows(const Plan& k, const f32x2* u, const f32x2* v, float* red, float* tot) {
  constexpr int W = 4 * NP;
  if ((int)threadIdx.x < k.rl * k.vpr) {
    ulonglong2* o = reinterpret_cast<ulonglong2*>(red + threadIdx.x * W);
    if constexpr (NP == 1) {
      o[0] = make_ulonglong2(u[0], v[0]);
    } else {
#pragma unroll
      for (int e = 0; e < NP / 2; ++e) {
        o[e] = make_ulonglong2(u[2 * e], u[2 * e + 1]);
        o[NP / 2 + e] = make_ulonglong2(v[2 * e], v[2 * e + 1]);
      }
    }
  }
  __syncthreads();
  const int n = k.vpr * W;
  for (int i = threadIdx.x; i < n; i += kNT) {
    float a = 0.f;
#pragma unroll 8
    for (int r = 0; r < k.rl; ++r) a += red[r * n + i];
    tot[i] = a;
  }
  __syncthreads();
}

// A group's sums are taken by `seg` neighbouring lanes, a power of two that
// covers its D channels or a warp.
__device__ __forceinline__ int lanes_of_group(int D) {
  int seg = 1;
  while (seg < D && seg < 32) seg *= 2;
  return seg;
}
__device__ __forceinline__ float group_sum(float a, int seg) {
  for (int o = seg >> 1; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  return a;
}

// V values of a per-channel tensor; one read where the base is aligned
template <typename T, int V>
__device__ __forceinline__ void load_channels(const T* base, int c, float none, f32x2* o) {
  constexpr int NP = Vecs<T, V>::NP;
  if (!base) {
#pragma unroll
    for (int e = 0; e < NP; ++e) o[e] = both(none);
  } else if (V > 1 && reinterpret_cast<uintptr_t>(base) % sizeof(typename Vecs<T, V>::word) == 0) {
    Vecs<T, V>::unpack(*reinterpret_cast<const typename Vecs<T, V>::word*>(base + c), o);
  } else {
#pragma unroll
    for (int e = 0; e < NP; ++e) o[e] = pack_f32x2(ld(base + c + 2 * e), 2 * e + 1 < V ? ld(base + c + 2 * e + 1) : 0.f);
  }
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
__global__ void __launch_bounds__(kNT, 3)
fwd_kernel(Norm g, Plan k, const T* __restrict__ x, const T* __restrict__ gamma, const T* __restrict__ beta,
           T* __restrict__ y, float* __restrict__ mean_out, float* __restrict__ rstd_out, Act8 x8) {
  typedef typename Vecs<T, V>::word word;
  constexpr int NP = Vecs<T, V>::NP;
  extern __shared__ __align__(16) unsigned char sm[];
  cg::cluster_group cluster = cg::this_cluster();
  const Place p = place_of<V>(g, k);
  word* const data = reinterpret_cast<word*>(sm);
  constexpr int W = 4 * NP;
  float* const red = reinterpret_cast<float*>(sm + k.data_bytes);
  float* const tot = red + kNT * W;
  float* const base = tot + k.vpr * W;                                    // what the sums are about, per channel
  float2* const part = reinterpret_cast<float2*>(base + k.vpr * 2 * NP);  // (mean, squares) of the block's groups
  float2* const stat = part + k.groups;                                   // (mean, rstd) of the slab's

  // read, sum, keep
  f32x2 s[NP], d[NP], q[NP];
#pragma unroll
  for (int e = 0; e < NP; ++e) s[e] = d[e] = q[e] = 0;
  int gi[V];
  groups_of<V>(g.D, min(p.vl * V, p.S - 1), gi);
  const T* xp = x + (p.row0 + p.r) * g.xs + g.xo + p.c;
  uint8_t* cp = KEEP != kSrcFull ? x8.codes + (p.row0 + p.r) * g.C + p.c : nullptr;
  float* scp = KEEP != kSrcFull ? x8.scales + (p.row0 + p.r) * x8.nblk + (p.c >> x8.shift) : nullptr;
  const bool scaler = KEEP != kSrcFull && (p.c & ((1 << x8.shift) - 1)) == 0;
  const int64_t xstep = k.rl * g.xs;
  const int left = p.on ? p.rows - p.r : 0;  // rows from this lane's first on
  // sums about the share's first row: one value per channel, the same for every row lane
  if (p.on && p.rows > 0) {
    Vecs<T, V>::unpack(*reinterpret_cast<const word*>(x + p.row0 * g.xs + g.xo + p.c), s);
    if (p.r == 0) {
#pragma unroll
      for (int e = 0; e < NP; ++e) *reinterpret_cast<f32x2*>(base + p.vl * 2 * NP + 2 * e) = s[e];
    }
#pragma unroll
    for (int e = 0; e < NP; ++e) s[e] = neg(s[e]);
  }
  word* dp = data + p.r * k.vpr + p.vl;
  const int dstep = k.rl * k.vpr;
  constexpr int kAhead = V == 1 ? 8 : 4;  // rows in flight
  for (int r0 = 0; r0 < p.rows; r0 += kAhead * k.rl) {
    word w[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a, xp += xstep) {
      w[a] = word{};
      if (r0 + a * k.rl < left) w[a] = *reinterpret_cast<const word*>(xp);
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const bool in = r0 + a * k.rl < left;
      f32x2 f[NP];
      Vecs<T, V>::unpack(w[a], f);
      if (in) {
        *dp = w[a];
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          const f32x2 t = add_f32x2(f[e], s[e]);
          d[e] = add_f32x2(d[e], t);
          fma_f32x2(q[e], t, t);
        }
      }
      dp += dstep;
      if (KEEP != kSrcFull) {  // lanes of a block of channels are neighbours; those without data bring zeros
        const uint32_t m = block_max<T, V>(w[a], (1 << x8.shift) / V);
        if (in) {
          float inv;
          const float sc = scale_of<KEEP>(m, &inv);
          *reinterpret_cast<typename Word<V>::type*>(cp) = pack_codes<KEEP, V>(f, inv);
          if (scaler) *scp = sc;
        }
        cp += (int64_t)k.rl * g.C;
        scp += (int64_t)k.rl * x8.nblk;
      }
    }
  }

  // the block's mean and squares of each group, from those of its channels
  const int groups = p.S / g.D, seg = lanes_of_group(g.D);
  join_rows<NP>(k, d, q, red, tot);
  {
    const float n = (float)p.rows, in = p.rows > 0 ? 1.f / n : 0.f;
    auto channel = [&](int c, float* mean, float* squares) {
      const int vl = c / V, e = c - vl * V;
      const float sd = tot[vl * W + e], sq = tot[vl * W + 2 * NP + e], t = sq - sd * sd * in;
      *mean = base[vl * 2 * NP + e] + sd * in;
      *squares = t < 0.f ? 0.f : t;  // NaN stays
    };
    for (int i0 = 0; i0 < groups; i0 += kNT / seg) {
      const int i = i0 + (int)threadIdx.x / seg, l = threadIdx.x & (seg - 1);
      const bool in_slice = i < groups && p.rows > 0;
      float a = 0.f, m, sq;
      for (int c = l; c < g.D && in_slice; c += seg) {
        channel(i * g.D + c, &m, &sq);
        a += m;
      }
      const float mean = group_sum(a, seg) / (float)g.D;
      a = 0.f;
      for (int c = l; c < g.D && in_slice; c += seg) {
        channel(i * g.D + c, &m, &sq);
        a += fmaf(n * (m - mean), m - mean, sq);
      }
      a = group_sum(a, seg);
      if (l == 0 && i < groups) part[i] = make_float2(mean, a);
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
    f32x2 ga[NP], be[NP], mu[NP], rs[NP];
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      const float2 a = stat[gi[2 * e]], b = stat[gi[2 * e + 1 < V ? 2 * e + 1 : 2 * e]];
      mu[e] = pack_f32x2(-a.x, -b.x);
      rs[e] = pack_f32x2(a.y, b.y);
    }
    load_channels<T, V>(gamma, p.c, 1.f, ga);
    load_channels<T, V>(beta, p.c, 0.f, be);
    T* yp = y + (p.row0 + p.r) * g.ys + g.yo + p.c;
    const int64_t ystep = k.rl * g.ys;
    dp = data + p.r * k.vpr + p.vl;
#pragma unroll 2
    for (int r = p.r; r < p.rows; r += k.rl, yp += ystep, dp += dstep) {
      f32x2 f[NP];
      Vecs<T, V>::unpack(*dp, f);
#pragma unroll
      for (int e = 0; e < NP; ++e)
        f[e] = add_apart(mul_f32x2(mul_f32x2(add_f32x2(f[e], mu[e]), rs[e]), ga[e]), be[e]);
      act_p<NP>(g.act, f);
      *reinterpret_cast<word*>(yp) = Vecs<T, V>::pack(f);
    }
  }
  if (k.cl > 1) cluster_wait();  // no block leaves while another reads its sums
}

template <typename T, int V, int SRC>
__global__ void __launch_bounds__(kNT, 2)
bwd_kernel(Norm g, Plan k, const T* __restrict__ x, Act8 x8, const T* __restrict__ gy, const T* __restrict__ gamma,
           const T* __restrict__ beta, const float* __restrict__ mean, const float* __restrict__ rstd,
           T* __restrict__ gx, float2* __restrict__ sums) {
  typedef typename Vecs<T, V>::word word;
  typedef typename Word<SRC == kSrcFull ? V * (int)sizeof(T) : V>::type xword;
  constexpr int NP = Vecs<T, V>::NP;
  extern __shared__ __align__(16) unsigned char sm[];
  cg::cluster_group cluster = cg::this_cluster();
  const Place p = place_of<V>(g, k);
  word* const gdata = reinterpret_cast<word*>(sm);
  xword* const xdata = reinterpret_cast<xword*>(sm + (size_t)k.rows * k.vpr * sizeof(word));
  constexpr int W = 4 * NP;
  float* const red = reinterpret_cast<float*>(sm + k.data_bytes);
  float* const tot = red + kNT * W;                                       // sums of du and of du * xh per channel
  float2* const part = reinterpret_cast<float2*>(tot + k.vpr * W);        // (s1, s2) of the block's groups
  float2* const stat = part + k.groups;                                   // of the slab's, over the count

  int gi[V];
  groups_of<V>(g.D, min(p.vl * V, p.S - 1), gi);
  f32x2 ga[NP], be[NP], mu[NP], rs[NP];
#pragma unroll
  for (int e = 0; e < NP; ++e) ga[e] = be[e] = mu[e] = rs[e] = 0;
  if (p.on) {
    load_channels<T, V>(gamma, p.c, 1.f, ga);
    load_channels<T, V>(beta, p.c, 0.f, be);
    const int64_t at = p.n * g.G + p.c0 / g.D;
    const float m0 = -__ldg(mean + at + gi[0]), r0 = __ldg(rstd + at + gi[0]);
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      mu[e] = both(m0);
      rs[e] = both(r0);
    }
    if (gi[0] != gi[V - 1]) {
#pragma unroll
      for (int e = 0; e < NP; ++e) {
        const int i = gi[2 * e], j = gi[2 * e + 1 < V ? 2 * e + 1 : 2 * e];
        mu[e] = pack_f32x2(-__ldg(mean + at + i), -__ldg(mean + at + j));
        rs[e] = pack_f32x2(__ldg(rstd + at + i), __ldg(rstd + at + j));
      }
    }
  }
  const T* gp = gy + (p.row0 + p.r) * g.ys + g.yo + p.c;
  const int64_t gstep = k.rl * g.ys;
  // x and its scale, one row lane's step at a time
  const int64_t first = p.row0 + p.r;
  const xword* xp;
  int64_t xstep;
  if constexpr (SRC == kSrcFull) {
    xp = reinterpret_cast<const xword*>(x + first * g.xs + g.xo + p.c);
    xstep = k.rl * g.xs / V;
  } else {
    xp = reinterpret_cast<const xword*>(x8.codes + first * g.C + p.c);
    xstep = (int64_t)k.rl * g.C / V;
  }
  const float* scp = SRC == kSrcFull ? nullptr : x8.scales + first * x8.nblk + (p.c >> x8.shift);
  const int64_t scstep = SRC == kSrcFull ? 0 : (int64_t)k.rl * x8.nblk;
  // xh and du of one vector, from what was stored
  auto eval = [&](word gw, xword xw, float sc, f32x2* xh, f32x2* du) {
    f32x2 t[NP];
    if constexpr (SRC == kSrcFull) {
      Vecs<T, V>::unpack(xw, xh);
    } else {
      unpack_codes<SRC, V>(xw, sc, xh);
    }
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      const f32x2 d = SRC == kSrcFull ? add_f32x2(xh[e], mu[e]) : add_apart(xh[e], mu[e]);
      xh[e] = mul_f32x2(d, rs[e]);
      t[e] = add_apart(mul_f32x2(xh[e], ga[e]), be[e]);
    }
    slope_p<NP>(g.act, t);
    Vecs<T, V>::unpack(gw, du);
#pragma unroll
    for (int e = 0; e < NP; ++e) du[e] = mul_f32x2(du[e], t[e]);
  };

  // read, sum, keep
  f32x2 a[NP], b[NP];
#pragma unroll
  for (int e = 0; e < NP; ++e) a[e] = b[e] = 0;
  const int at0 = p.r * k.vpr + p.vl, dstep = k.rl * k.vpr;
  if (p.on) {
    constexpr int kAhead = V == 1 ? 4 : 2;
    const float* sq = scp;
    int at = at0;
    for (int r0 = p.r; r0 < p.rows; r0 += kAhead * k.rl) {
      word gw[kAhead];
      xword xw[kAhead];
      float sc[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        gw[i] = word{};
        xw[i] = xword{};
        sc[i] = 0.f;
        if (r0 + i * k.rl < p.rows) {
          gw[i] = *reinterpret_cast<const word*>(gp);
          xw[i] = *xp;
          if (SRC != kSrcFull) sc[i] = __ldg(sq);
        }
        gp += gstep;
        xp += xstep;
        sq += scstep;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (r0 + i * k.rl >= p.rows) break;
        gdata[at] = gw[i];
        xdata[at] = xw[i];
        at += dstep;
        f32x2 xh[NP], du[NP];
        eval(gw[i], xw[i], sc[i], xh, du);
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          a[e] = add_f32x2(a[e], du[e]);
          fma_f32x2(b[e], du[e], xh[e]);
        }
      }
    }
  }
  join_rows<NP>(k, a, b, red, tot);
  const int groups = p.S / g.D, seg = lanes_of_group(g.D);
  for (int i0 = 0; i0 < groups; i0 += kNT / seg) {
    const int i = i0 + (int)threadIdx.x / seg, l = threadIdx.x & (seg - 1);
    float s1 = 0.f, s2 = 0.f;
    for (int c = l; c < g.D && i < groups; c += seg) {
      const int ch = i * g.D + c, vl = ch / V, e = ch - vl * V;
      const float w = gamma ? ld(gamma + p.c0 + ch) : 1.f;
      s1 = fmaf(w, tot[vl * W + e], s1);
      s2 = fmaf(w, tot[vl * W + 2 * NP + e], s2);
    }
    s1 = group_sum(s1, seg);
    s2 = group_sum(s2, seg);
    if (l == 0 && i < groups) part[i] = make_float2(s1, s2);
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
      const float* o = cluster.map_shared_rank(tot, j) + c / V * W + c % V;
      s1 += o[0];
      s2 += o[2 * NP];
    }
    sums[p.n * g.C + p.c0 + c] = make_float2(s1, s2);
  }
  __syncthreads();
  if (k.cl > 1) cluster_arrive();

  // write: gx = du * (gamma rstd) - rstd s1 - xh * (rstd s2)
  if (gx && p.on) {
    f32x2 c1[NP], c2[NP], c3[NP];
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      const float2 u = stat[gi[2 * e]], v = stat[gi[2 * e + 1 < V ? 2 * e + 1 : 2 * e]];
      c1[e] = mul_f32x2(ga[e], rs[e]);
      c2[e] = neg(mul_f32x2(pack_f32x2(u.x, v.x), rs[e]));
      c3[e] = neg(mul_f32x2(pack_f32x2(u.y, v.y), rs[e]));
    }
    T* op = gx + first * g.xs + g.xo + p.c;
    const int64_t ostep = k.rl * g.xs;
    int at = at0;
    for (int r = p.r; r < p.rows; r += k.rl, op += ostep, scp += scstep, at += dstep) {
      f32x2 xh[NP], du[NP];
      eval(gdata[at], xdata[at], SRC == kSrcFull ? 0.f : __ldg(scp), xh, du);
#pragma unroll
      for (int e = 0; e < NP; ++e) du[e] = fma2(du[e], c1[e], fma2(xh[e], c3[e], c2[e]));
      *reinterpret_cast<word*>(op) = Vecs<T, V>::pack(du);
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
