// Channels-last group norm, forward and backward: the slab kernels, which
// read their inputs once, and the stream kernels, which read them twice.
//
// A slab is one sample's pixels times a slice of channels that holds whole
// groups, at least one 128-byte line wide where the channels allow it. A
// cluster of thread blocks owns a slab, each block a share of its pixels: it
// reads them once, takes the sums on the way and leaves the data as read in
// shared memory; the blocks join their sums through the cluster's distributed
// shared memory; then each writes its outputs from its own shared memory.
// Bytes moved are the floor's: inputs once, outputs once. The forward also
// writes the 8-bit checkpoint of x from the registers that hold it (a block
// of channels is a few neighbouring lanes).
//
// Slabs that no cluster of eight blocks can hold are streamed: one launch
// leaves the sums of each chunk of pixels in the workspace, a second reads
// the inputs again (from L2 where they fit it; it walks the chunks last to
// first, to begin with what the first launch left there), joins the chunks'
// sums for its groups and writes the outputs. The same code in three modes.
//
// The variance is not taken from sums of squares of x: a block sums x - s and
// (x - s)^2 about one value s per channel, turns them into a mean and squares
// about that mean, and joins channels and blocks by the parallel form of the
// two (see norm.cu). s is the middle one of the values of three of the block's
// pixels: the sums lose what s is away from the rest, squared, so no single
// pixel may decide it. The three lie at multiples of the golden section, which
// no width of an image puts into one of its columns. Every order is fixed.
//
// Arithmetic is on pairs of channels (the two lanes of the packed fp32
// instructions). Rows are fetched by asynchronous copies, a batch ahead.
// What bounds the kernels is latency with few warps and a block's fixed cost:
// issue is active 53 to 61 % of the time and DRAM 18 to 21 %, a fifth of the
// warps' time are fixed waits and a tenth to a sixth shared memory's, the last
// wave of blocks is part full, and about 900 instructions per warp are a
// block's start, joins and cluster barrier. 64x56x56x128 bf16, 32 groups, SiLU
// takes 49 us forward with its checkpoint (2.7 TB/s of the floor's bytes) and
// 65 backward from it (2.0), 29.0 and 37.3 M warp instructions; 64x28x28x256
// bf16, 16 groups, ReLU 31 us backward (2.4 TB/s). Streamed, 2x256x256x64 fp32 takes 13 + 15 us (the
// second read comes from L2). Sums per thread instead of about the block's
// first pixel need a second join (9 us more for the step).
#pragma once

#include <cooperative_groups.h>

#include "norm.cuh"
#include "norm_slab.h"

namespace dwconv {
namespace norm {
namespace slab {

namespace cg = cooperative_groups;

enum Mode : int { kSlab = 0, kSums = 1, kApply = 2 };

template <int BYTES> struct Word;
template <> struct Word<16> { typedef uint4 type; };
template <> struct Word<8> { typedef uint2 type; };
template <> struct Word<4> { typedef uint32_t type; };

// Asynchronous copies into the thread's own slots: no thread reads another's,
// so a thread waits for its own copies only.
template <typename W>
__device__ __forceinline__ void copy_async(W* dst, const void* src) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  if constexpr (sizeof(W) == 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  } else {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"((int)sizeof(W)) : "memory");
  }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// two 16-bit values as a pair, exact
template <typename T>
__device__ __forceinline__ f32x2 pair_of(uint32_t u) {
  if constexpr (std::is_same<T, __half>::value) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
    return pack_f32x2(f.x, f.y);
  } else {
    return pack_f32x2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
}
template <typename T>
__device__ __forceinline__ uint32_t word_of(f32x2 v) {
  float a, b;
  unpack_f32x2(v, a, b);
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// the middle one of three values, or of three pairs of 16-bit values
template <typename T>
__device__ __forceinline__ uint32_t middle_word(uint32_t a, uint32_t b, uint32_t c) {
  if constexpr (sizeof(T) == 4) {
    const float x = __uint_as_float(a), y = __uint_as_float(b);
    return __float_as_uint(fmaxf(fminf(x, y), fminf(fmaxf(x, y), __uint_as_float(c))));
  } else {
    typedef typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type P;
    const P x = *reinterpret_cast<const P*>(&a), y = *reinterpret_cast<const P*>(&b), z = *reinterpret_cast<const P*>(&c);
    const P m = __hmax2(__hmin2(x, y), __hmin2(__hmax2(x, y), z));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
}

// A thread's V channels of a row, as stored (word) and as pairs. n: how many
// of them exist (side by side: V or none).
template <typename T, int V, bool STR>
struct Lay {
  typedef typename Word<V * (int)sizeof(T)>::type word;
  typedef typename Word<V>::type codes;
  static constexpr int NP = V / 2;

  static __device__ __forceinline__ word load(const T* p, int vpr, int n) {
    word w{};
    if constexpr (STR) {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < n) reinterpret_cast<T*>(&w)[e] = p[e * vpr];
    } else {
      if (n > 0) w = *reinterpret_cast<const word*>(p);
    }
    return w;
  }
  // the same, into shared memory; side by side it only begins the copy
  static __device__ __forceinline__ void fetch(word* dst, const T* p, int vpr, int n) {
    if constexpr (STR) {
      *dst = load(p, vpr, n);
    } else {
      copy_async(dst, p);
    }
  }
  static __device__ __forceinline__ void fetch_codes(codes* dst, const uint8_t* p, int vpr, int n) {
    if constexpr (STR) {
      *dst = load_codes(p, vpr, n);
    } else {
      copy_async(dst, p);
    }
  }
  static __device__ __forceinline__ void store(T* p, int vpr, int n, word w) {
    if constexpr (STR) {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < n) p[e * vpr] = reinterpret_cast<const T*>(&w)[e];
    } else {
      if (n > 0) *reinterpret_cast<word*>(p) = w;
    }
  }
  static __device__ __forceinline__ codes load_codes(const uint8_t* p, int vpr, int n) {
    codes w{};
    if constexpr (STR) {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < n) reinterpret_cast<uint8_t*>(&w)[e] = p[e * vpr];
    } else {
      if (n > 0) w = *reinterpret_cast<const codes*>(p);
    }
    return w;
  }
  static __device__ __forceinline__ void unpack(word w, f32x2* f) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(&w);
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      if constexpr (sizeof(T) == 4) {
        f[e] = pack_f32x2(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1]));
      } else {
        f[e] = pair_of<T>(u[e]);
      }
    }
  }
  static __device__ __forceinline__ word pack(const f32x2* f) {
    word w;
    uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      if constexpr (sizeof(T) == 4) {
        float a, b;
        unpack_f32x2(f[e], a, b);
        u[2 * e] = __float_as_uint(a);
        u[2 * e + 1] = __float_as_uint(b);
      } else {
        u[e] = word_of<T>(f[e]);
      }
    }
    return w;
  }
  // per channel the middle one of three values; of a NaN and two others, one of those
  static __device__ __forceinline__ word middle(word a, word b, word c) {
    word w;
    const uint32_t *ua = reinterpret_cast<const uint32_t*>(&a), *ub = reinterpret_cast<const uint32_t*>(&b),
                   *uc = reinterpret_cast<const uint32_t*>(&c);
    uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int e = 0; e < (int)sizeof(word) / 4; ++e) u[e] = middle_word<T>(ua[e], ub[e], uc[e]);
    return w;
  }
  // V values of a per-channel tensor from channel c
  static __device__ __forceinline__ void channels(const T* base, int c, int vpr, int n, float none, f32x2* o) {
    if (!base) {
#pragma unroll
      for (int e = 0; e < NP; ++e) o[e] = both(none);
    } else if (!STR && reinterpret_cast<uintptr_t>(base) % sizeof(word) == 0) {
      unpack(load(base + c, vpr, n), o);
    } else {
      word w{};
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (e < n) reinterpret_cast<T*>(&w)[e] = base[c + (STR ? e * vpr : e)];
      unpack(w, o);
    }
  }
};

// The scales of V codes: one where they lie side by side.
template <int V, bool STR>
struct Scales {
  static constexpr int n = STR ? V : 1;
  float s[n];
  static __device__ __forceinline__ void fetch(Scales* dst, const Act8& t, int64_t row, int c, int vpr, int nv) {
    const float* p = t.scales + row * t.nblk;
    if constexpr (STR) {
#pragma unroll
      for (int e = 0; e < V; ++e) dst->s[e] = e < nv ? __ldg(p + ((c + e * vpr) >> t.shift)) : 0.f;
    } else {
      copy_async(&dst->s[0], p + (c >> t.shift));
    }
  }
};
template <int SRC, int V, bool STR, typename W>
__device__ __forceinline__ void values_of(W w, const Scales<V, STR>& sc, f32x2* f) {
  const uint32_t* u = reinterpret_cast<const uint32_t*>(&w);
#pragma unroll
  for (int h = 0; h < V / 4; ++h) {
    decode4<SRC>(u[h], STR ? 1.f : sc.s[0], f + 2 * h);
    if constexpr (STR) {
      f[2 * h] = mul_f32x2(f[2 * h], pack_f32x2(sc.s[4 * h], sc.s[4 * h + 1]));
      f[2 * h + 1] = mul_f32x2(f[2 * h + 1], pack_f32x2(sc.s[4 * h + 2], sc.s[4 * h + 3]));
    }
  }
}

template <int SRC, int V>
__device__ __forceinline__ typename Word<V>::type pack_codes(const f32x2* f, float inv) {
  typename Word<V>::type w;
  uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
  for (int h = 0; h < V / 4; ++h) u[h] = encode4<SRC>(f[2 * h], f[2 * h + 1], inv);
  return w;
}

// Sums two vectors over the block's row lanes, in lane order. Afterwards
// tot[vl * 4 NP + e] is the sum of u's element e of vector vl of the slice
// and tot[vl * 4 NP + 2 NP + e] that of v's. red holds kNT * 4 NP floats.
template <int NP>
__device__ __forceinline__ void join_rows(const Plan& k, const f32x2* u, const f32x2* v, float* red, float* tot) {
  constexpr int W = 4 * NP;
  if ((int)threadIdx.x < k.rl * k.vpr) {
    ulonglong2* o = reinterpret_cast<ulonglong2*>(red + threadIdx.x * W);
#pragma unroll
    for (int e = 0; e < NP / 2; ++e) {
      o[e] = make_ulonglong2(u[2 * e], u[2 * e + 1]);
      o[NP / 2 + e] = make_ulonglong2(v[2 * e], v[2 * e + 1]);
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

// where channel c of the slice lies in a table of W floats per vector
template <int V, bool STR, int W>
__device__ __forceinline__ int table_at(const Plan& k, int c) {
  const int q = STR ? (int)k.d_vpr.div((uint32_t)c) : c / V;
  return STR ? (c - q * k.vpr) * W + q : q * W + (c - q * V);
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

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync(int blocks) {
  if (blocks == 1) {
    __syncthreads();
  } else {
    cluster_arrive();
    cluster_wait();
  }
}

struct Place {
  int64_t n, row0;   // sample, first row of the block in the tensor
  int part, rows;    // block of the slab, its rows (0: none)
  int c0, S;         // first channel and channels of the slice
  int g0, groups;    // first group and groups of it
  int c, vl, r;      // this thread's first channel, vector and row lane
  int nv;            // its channels that exist
};

template <int V, bool STR>
__device__ __forceinline__ Place place_of(const Norm& g, const Plan& k, uint32_t block) {
  Place p;
  uint32_t unit, n, r;
  p.part = (int)k.d_parts.divmod(block, unit);
  const int slice = (int)k.d_slices.divmod(unit, n);
  p.n = n;
  p.c0 = slice * k.S;
  p.g0 = slice * k.groups;
  p.S = min(k.S, g.C - p.c0);
  p.groups = p.S == k.S ? k.groups : (int)k.d_D.div((uint32_t)p.S);
  const int64_t r0 = (int64_t)p.part * k.rows;
  p.rows = (int)(r0 < g.P ? (g.P - r0 < k.rows ? g.P - r0 : k.rows) : 0);
  p.row0 = p.n * g.P + r0;
  p.vl = (int)k.d_vpr.divmod(threadIdx.x, r);
  p.r = (int)r;
  p.c = p.c0 + (STR ? p.vl : p.vl * V);
  if (p.r >= k.rl) {
    p.nv = 0;
  } else if (STR) {
    p.nv = p.vl < p.S ? min((int)k.d_vpr.div((uint32_t)(p.S - p.vl + k.vpr - 1)), V) : 0;
  } else {
    p.nv = p.vl * V < p.S ? V : 0;
  }
  return p;
}

// group of the slice that each of a thread's channels belongs to (0 for those that do not exist)
template <int V, bool STR>
__device__ __forceinline__ void groups_of(const Norm& g, const Plan& k, const Place& p, int* gi) {
  if (STR) {
#pragma unroll
    for (int e = 0; e < V; ++e) gi[e] = e < p.nv ? (int)k.d_D.div((uint32_t)(p.vl + e * k.vpr)) : 0;
  } else {
    const int first = p.nv > 0 ? p.vl * V : 0;
    uint32_t uq;
    int r = (int)k.d_D.divmod((uint32_t)first, uq), q = (int)uq;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      gi[e] = q;
      if (++r == g.D) {
        r = 0;
        ++q;
      }
    }
  }
}

// rows of part j of a slab
__device__ __forceinline__ float rows_of(const Norm& g, const Plan& k, int j) {
  const int64_t left = g.P - (int64_t)j * k.rows;
  return (float)(left >= k.rows ? k.rows : left > 0 ? (int)left : 0);
}

template <typename T, int V, bool STR, int KEEP, int MODE>
__global__ void __launch_bounds__(kNT, 3)
fwd_kernel(Norm g, Plan k, const T* __restrict__ x, const T* __restrict__ gamma, const T* __restrict__ beta,
           T* __restrict__ y, float* __restrict__ mean_out, float* __restrict__ rstd_out, Act8 x8,
           float2* __restrict__ gsums) {
  typedef Lay<T, V, STR> L;
  typedef typename L::word word;
  constexpr int NP = L::NP, W = 4 * NP;
  extern __shared__ __align__(16) unsigned char sm[];
  const Place p = place_of<V, STR>(g, k, MODE == kApply ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  word* const data = reinterpret_cast<word*>(sm);
  float* const red = reinterpret_cast<float*>(sm + k.data_bytes);
  float* const tot = red + kNT * W;
  float* const base = tot + k.vpr * W;                               // what the sums are about, per channel
  float2* const part = reinterpret_cast<float2*>(base + k.vpr * V);  // (mean, squares) of the block's groups
  float2* const stat = part + k.groups;                              // (mean, rstd) of the slab's
  const int groups = p.groups;
  int gi[V];
  groups_of<V, STR>(g, k, p, gi);
  const T* xp = x + (p.row0 + p.r) * g.xs + g.xo + p.c;
  const int64_t xstep = k.rl * g.xs;
  const int at0 = p.r * k.vpr + p.vl, dstep = k.rl * k.vpr;
  // Rows p.r + j * rl of the share, j < mine, are this thread's. They come in batches of kBatch, a batch ahead of the one
  // in use; a slab keeps every row, a stream has slots for two batches.
  const int mine = p.nv > 0 && p.r < p.rows ? (p.rows - p.r + k.rl - 1) / k.rl : 0;
  const int batches = ((p.rows + k.rl - 1) / k.rl + kBatch - 1) / kBatch;
  auto slot = [&](int j) { return MODE == kSlab ? at0 + j * dstep : (j & (2 * kBatch - 1)) * kNT + (int)threadIdx.x; };
  auto fetch = [&](int b) {
#pragma unroll
    for (int a = 0; a < kBatch; ++a, xp += xstep) {
      const int j = b * kBatch + a;
      if (j < mine) L::fetch(data + slot(j), xp, k.vpr, p.nv);
    }
    copies_commit();
  };
  fetch(0);
  fetch(1);
  if (MODE != kApply) dependents_may_start();
  if (p.nv > 0) {  // needed after the barriers
    if (gamma) prefetch_l2(gamma + p.c);
    if (beta) prefetch_l2(beta + p.c);
  }

  if constexpr (MODE != kApply) {
    // read, sum, keep
    f32x2 s[NP], d[NP], q[NP];
#pragma unroll
    for (int e = 0; e < NP; ++e) s[e] = d[e] = q[e] = 0;
    if (p.rows > 0) {  // one value per channel, the same for every row lane
      const T* const rows = x + p.row0 * g.xs + g.xo + p.c;
      auto pixel = [&](uint32_t part) {  // at part / 2^32 of the share
        return L::load(rows + (int64_t)__umulhi((uint32_t)p.rows, part) * g.xs, k.vpr, p.nv);
      };
      L::unpack(L::middle(pixel(0x3c6ef372u), pixel(0x9e3779b9u), pixel(0xdaa66d2bu)), s);
      if (p.r == 0) {
#pragma unroll
        for (int e = 0; e < NP; ++e) *reinterpret_cast<f32x2*>(base + p.vl * V + 2 * e) = s[e];
      }
#pragma unroll
      for (int e = 0; e < NP; ++e) s[e] = neg(s[e]);
    }
    uint8_t* cp = KEEP != kSrcFull ? x8.codes + (p.row0 + p.r) * g.C + p.c : nullptr;
    float* scp = KEEP != kSrcFull ? x8.scales + (p.row0 + p.r) * x8.nblk + (p.c >> x8.shift) : nullptr;
    const bool scaler = KEEP != kSrcFull && (p.c & ((1 << x8.shift) - 1)) == 0;
    for (int b = 0; b < batches; ++b) {
      copies_wait<1>();
#pragma unroll
      for (int a = 0; a < kBatch; ++a) {
        const int j = b * kBatch + a;
        const bool in = j < mine;
        word w{};
        if (in) w = data[slot(j)];
        if (in) {
          f32x2 f[NP];
          L::unpack(w, f);
#pragma unroll
          for (int e = 0; e < NP; ++e) {
            const f32x2 t = add_f32x2(f[e], s[e]);
            d[e] = add_f32x2(d[e], t);
            fma_f32x2(q[e], t, t);
          }
        }
        if constexpr (KEEP != kSrcFull) {  // lanes of a block of channels are neighbours; those without data bring zeros
          const uint32_t m = block_max<T, V>(w, (1 << x8.shift) / V);
          if (in) {
            float inv;
            const float sc = scale_of<KEEP>(m, &inv);
            f32x2 f[NP];
            L::unpack(w, f);
            *reinterpret_cast<typename L::codes*>(cp) = pack_codes<KEEP, V>(f, inv);
            if (scaler) *scp = sc;
          }
          cp += (int64_t)k.rl * g.C;
          scp += (int64_t)k.rl * x8.nblk;
        }
      }
      fetch(b + 2);
    }

    // the block's mean and squares of each group, from those of its channels
    const int seg = lanes_of_group(g.D);
    join_rows<NP>(k, d, q, red, tot);
    const float n = (float)p.rows, in = p.rows > 0 ? 1.f / n : 0.f;
    auto channel = [&](int c, float* mean, float* squares) {
      const int i = table_at<V, STR, W>(k, c);
      const float sd = tot[i], t = tot[i + 2 * NP] - sd * sd * in;
      *mean = base[table_at<V, STR, V>(k, c)] + sd * in;
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
      const float mean = group_sum(a, seg) * k.inv_D;
      a = 0.f;
      for (int c = l; c < g.D && in_slice; c += seg) {
        channel(i * g.D + c, &m, &sq);
        a += fmaf(n * (m - mean), m - mean, sq);
      }
      a = group_sum(a, seg);
      if (l == 0 && i < groups) {
        if (MODE == kSlab) part[i] = make_float2(mean, a);
        else gsums[(p.n * k.parts + p.part) * g.G + p.g0 + i] = make_float2(mean, a);
      }
    }
    if constexpr (MODE == kSums) return;
  }

  // the slab's mean and rstd from its parts'
  auto finish = [&](int i, float mean, float sq) {
    const float rstd = 1.f / sqrtf(sq / k.total + g.eps);
    stat[i] = make_float2(mean, rstd);
    if (p.part == 0) {
      const int64_t at = p.n * g.G + p.g0 + i;
      if (mean_out) mean_out[at] = mean;
      if (rstd_out) rstd_out[at] = rstd;
    }
  };
  if constexpr (MODE == kSlab) {
    cluster_sync(k.parts);
    cg::cluster_group cluster = cg::this_cluster();
    // a lane per block of the cluster, eight lanes per group
    const int b = threadIdx.x & 7;
    const float n = b < k.parts ? rows_of(g, k, b) * (float)g.D : 0.f;
    for (int i0 = 0; i0 < groups; i0 += kNT / 8) {
      const int i = i0 + (int)threadIdx.x / 8;
      const bool in = i < groups && n > 0.f;
      const float2 v = in ? cluster.map_shared_rank(part, b)[i] : make_float2(0.f, 0.f);
      const float mean = group_sum(n * v.x, 8) / k.total;
      const float sq = group_sum(in ? fmaf(n * (v.x - mean), v.x - mean, v.y) : 0.f, 8);
      if (b == 0 && i < groups) finish(i, mean, sq);
    }
  } else {
    wait_for_previous();
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x >> 5; i < groups; i += kNT / 32) {
      const float2* o = gsums + p.n * k.parts * (int64_t)g.G + p.g0 + i;
      float2 v[kMaxParts / 32];  // every part's, read at once
#pragma unroll
      for (int h = 0; h < kMaxParts / 32; ++h)
        v[h] = lane + 32 * h < k.parts ? o[(int64_t)(lane + 32 * h) * g.G] : make_float2(0.f, 0.f);
      float a = 0.f, sq = 0.f;
#pragma unroll
      for (int h = 0; h < kMaxParts / 32; ++h) a = fmaf(rows_of(g, k, lane + 32 * h) * (float)g.D, v[h].x, a);
      const float mean = group_sum(a, 32) / k.total;
#pragma unroll
      for (int h = 0; h < kMaxParts / 32; ++h) {
        const float n = rows_of(g, k, lane + 32 * h) * (float)g.D;
        sq += n > 0.f ? fmaf(n * (v[h].x - mean), v[h].x - mean, v[h].y) : 0.f;
      }
      sq = group_sum(sq, 32);
      if (lane == 0) finish(i, mean, sq);
    }
  }
  __syncthreads();
  if (MODE == kSlab && k.parts > 1) cluster_arrive();  // this block has read the others' sums

  // write
  if (p.nv > 0) {
    f32x2 ga[NP], be[NP], mu[NP], rs[NP];
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      const float2 a = stat[gi[2 * e]], b = stat[gi[2 * e + 1]];
      mu[e] = pack_f32x2(-a.x, -b.x);
      rs[e] = pack_f32x2(a.y, b.y);
    }
    L::channels(gamma, p.c, k.vpr, p.nv, 1.f, ga);
    L::channels(beta, p.c, k.vpr, p.nv, 0.f, be);
    T* yp = y + (p.row0 + p.r) * g.ys + g.yo + p.c;
    const int64_t ystep = k.rl * g.ys;
    auto put = [&](word w) {
      f32x2 f[NP];
      L::unpack(w, f);
#pragma unroll
      for (int e = 0; e < NP; ++e)
        f[e] = add_apart(mul_f32x2(mul_f32x2(add_f32x2(f[e], mu[e]), rs[e]), ga[e]), be[e]);
      act_p<NP>(g.act, f);
      L::store(yp, k.vpr, p.nv, L::pack(f));
    };
    if constexpr (MODE == kSlab) {
#pragma unroll 2
      for (int j = 0; j < mine; ++j, yp += ystep) put(data[at0 + j * dstep]);
    } else {
      for (int b = 0; b < batches; ++b) {
        copies_wait<1>();
#pragma unroll
        for (int a = 0; a < kBatch; ++a, yp += ystep)
          if (b * kBatch + a < mine) put(data[slot(b * kBatch + a)]);
        fetch(b + 2);
      }
    }
  }
  if (MODE == kSlab && k.parts > 1) cluster_wait();  // no block leaves while another reads its sums
}

template <typename T, int V, bool STR, int SRC, int MODE>
__global__ void __launch_bounds__(kNT, V == 8 ? 2 : 3)
bwd_kernel(Norm g, Plan k, const T* __restrict__ x, Act8 x8, const T* __restrict__ gy, const T* __restrict__ gamma,
           const T* __restrict__ beta, const float* __restrict__ mean, const float* __restrict__ rstd,
           T* __restrict__ gx, Sums sums) {
  typedef Lay<T, V, STR> L;
  typedef typename L::word word;
  typedef Scales<V, STR> Scale;
  typedef typename std::conditional<SRC == kSrcFull, word, typename L::codes>::type xword;
  constexpr int NP = L::NP, W = 4 * NP;
  extern __shared__ __align__(16) unsigned char sm[];
  const Place p = place_of<V, STR>(g, k, MODE == kApply ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  word* const gdata = reinterpret_cast<word*>(sm);
  const int slots = MODE == kSlab ? k.rows * k.vpr : 2 * kBatch * kNT;
  xword* const xdata = reinterpret_cast<xword*>(gdata + slots);
  Scale* const sdata = reinterpret_cast<Scale*>(xdata + slots);  // a checkpoint's
  float* const red = reinterpret_cast<float*>(sm + k.data_bytes);
  float* const tot = red + kNT * W;                                 // sums of du and of du * xh per channel
  float2* const part = reinterpret_cast<float2*>(tot + k.vpr * W);  // (s1, s2) of the block's groups
  float2* const stat = part + k.groups;                             // of the slab's, over the count
  const int groups = p.groups;
  int gi[V];
  groups_of<V, STR>(g, k, p, gi);

  const int64_t first = p.row0 + p.r;
  const T* gp = gy + first * g.ys + g.yo + p.c;
  const int64_t gstep = k.rl * g.ys;
  const T* xp = SRC == kSrcFull ? x + first * g.xs + g.xo + p.c : nullptr;
  const int64_t xstep = k.rl * g.xs;
  const uint8_t* cp = SRC == kSrcFull ? nullptr : x8.codes + first * g.C + p.c;
  const int64_t cstep = (int64_t)k.rl * g.C;
  // rows and slots as in the forward
  const int at0 = p.r * k.vpr + p.vl, dstep = k.rl * k.vpr;
  const int mine = p.nv > 0 && p.r < p.rows ? (p.rows - p.r + k.rl - 1) / k.rl : 0;
  const int batches = ((p.rows + k.rl - 1) / k.rl + kBatch - 1) / kBatch;
  auto slot = [&](int j) { return MODE == kSlab ? at0 + j * dstep : (j & (2 * kBatch - 1)) * kNT + (int)threadIdx.x; };
  auto fetch = [&](int b) {
#pragma unroll
    for (int a = 0; a < kBatch; ++a) {
      const int j = b * kBatch + a;
      if (j < mine) {
        L::fetch(gdata + slot(j), gp, k.vpr, p.nv);
        if constexpr (SRC == kSrcFull) {
          L::fetch(xdata + slot(j), xp, k.vpr, p.nv);
        } else {
          L::fetch_codes(xdata + slot(j), cp, k.vpr, p.nv);
          Scale::fetch(sdata + slot(j), x8, first + (int64_t)j * k.rl, p.c, k.vpr, p.nv);
        }
      }
      gp += gstep;
      if constexpr (SRC == kSrcFull) xp += xstep;
      else cp += cstep;
    }
    copies_commit();
  };
  fetch(0);
  fetch(1);
  if (MODE != kApply) dependents_may_start();

  f32x2 ga[NP], be[NP], mu[NP], rs[NP];
  L::channels(gamma, p.c, k.vpr, p.nv, 1.f, ga);
  L::channels(beta, p.c, k.vpr, p.nv, 0.f, be);
  {
    const float* m = mean + p.n * g.G + p.g0;
    const float* r = rstd + p.n * g.G + p.g0;
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      mu[e] = both(-__ldg(m + gi[0]));
      rs[e] = both(__ldg(r + gi[0]));
    }
    if (STR || gi[0] != gi[V - 1]) {
#pragma unroll
      for (int e = 0; e < NP; ++e) {
        mu[e] = pack_f32x2(-__ldg(m + gi[2 * e]), -__ldg(m + gi[2 * e + 1]));
        rs[e] = pack_f32x2(__ldg(r + gi[2 * e]), __ldg(r + gi[2 * e + 1]));
      }
    }
  }
  // xh and du of one vector, from its slot
  auto eval = [&](int at, f32x2* xh, f32x2* du) {
    f32x2 t[NP];
    if constexpr (SRC == kSrcFull) {
      L::unpack(xdata[at], xh);
    } else {
      values_of<SRC, V, STR>(xdata[at], sdata[at], xh);
    }
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      const f32x2 d = SRC == kSrcFull ? add_f32x2(xh[e], mu[e]) : add_apart(xh[e], mu[e]);
      xh[e] = mul_f32x2(d, rs[e]);
      t[e] = add_apart(mul_f32x2(xh[e], ga[e]), be[e]);
    }
    slope_p<NP>(g.act, t);
    L::unpack(gdata[at], du);
#pragma unroll
    for (int e = 0; e < NP; ++e) du[e] = mul_f32x2(du[e], t[e]);
  };

  if constexpr (MODE != kApply) {
    // sum
    f32x2 a[NP], b[NP];
#pragma unroll
    for (int e = 0; e < NP; ++e) a[e] = b[e] = 0;
    for (int i = 0; i < batches; ++i) {
      copies_wait<1>();
#pragma unroll
      for (int h = 0; h < kBatch; ++h) {
        if (i * kBatch + h >= mine) break;
        f32x2 xh[NP], du[NP];
        eval(slot(i * kBatch + h), xh, du);
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          a[e] = add_f32x2(a[e], du[e]);
          fma_f32x2(b[e], du[e], xh[e]);
        }
      }
      fetch(i + 2);
    }
    join_rows<NP>(k, a, b, red, tot);
    const int seg = lanes_of_group(g.D);
    for (int i0 = 0; i0 < groups; i0 += kNT / seg) {
      const int i = i0 + (int)threadIdx.x / seg, l = threadIdx.x & (seg - 1);
      float s1 = 0.f, s2 = 0.f;
      for (int c = l; c < g.D && i < groups; c += seg) {
        const int ch = i * g.D + c, t = table_at<V, STR, W>(k, ch);
        const float w = gamma ? ld(gamma + p.c0 + ch) : 1.f;
        s1 = fmaf(w, tot[t], s1);
        s2 = fmaf(w, tot[t + 2 * NP], s2);
      }
      s1 = group_sum(s1, seg);
      s2 = group_sum(s2, seg);
      if (l == 0 && i < groups) {
        if (MODE == kSlab) part[i] = make_float2(s1, s2);
        else sums.groups[(p.n * k.parts + p.part) * g.G + p.g0 + i] = make_float2(s1, s2);
      }
    }
    if constexpr (MODE == kSums) {
      for (int c = threadIdx.x; c < p.S; c += kNT) {
        const int t = table_at<V, STR, W>(k, c);
        sums.channels[(p.n * k.parts + p.part) * g.C + p.c0 + c] = make_float2(tot[t], tot[t + 2 * NP]);
      }
      return;
    }
  }

  if constexpr (MODE == kSlab) {
    cluster_sync(k.parts);
    cg::cluster_group cluster = cg::this_cluster();
    // a lane per block of the cluster, eight lanes per group, then per channel of this block's share
    const int b = threadIdx.x & 7;
    for (int i0 = 0; i0 < groups; i0 += kNT / 8) {
      const int i = i0 + (int)threadIdx.x / 8;
      const float2 v = i < groups && b < k.parts ? cluster.map_shared_rank(part, b)[i] : make_float2(0.f, 0.f);
      const float s1 = group_sum(v.x, 8), s2 = group_sum(v.y, 8);
      if (b == 0 && i < groups) stat[i] = make_float2(s1 * k.inv_total, s2 * k.inv_total);
    }
    const int share = (int)k.d_parts.div((uint32_t)(p.S + k.parts - 1)), lo = p.part * share, hi = min(lo + share, p.S);
    for (int c0 = lo; c0 < hi; c0 += kNT / 8) {
      const int c = c0 + (int)threadIdx.x / 8;
      float s1 = 0.f, s2 = 0.f;
      if (c < hi && b < k.parts) {
        const float* o = cluster.map_shared_rank(tot, b) + table_at<V, STR, W>(k, c);
        s1 = o[0];
        s2 = o[2 * NP];
      }
      s1 = group_sum(s1, 8);
      s2 = group_sum(s2, 8);
      if (b == 0 && c < hi) sums.channels[p.n * g.C + p.c0 + c] = make_float2(s1, s2);
    }
  } else {
    wait_for_previous();
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x >> 5; i < groups; i += kNT / 32) {
      const float2* o = sums.groups + p.n * k.parts * (int64_t)g.G + p.g0 + i;
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int h = 0; h < kMaxParts / 32; ++h) {
        if (lane + 32 * h >= k.parts) continue;
        const float2 v = o[(int64_t)(lane + 32 * h) * g.G];
        s1 += v.x;
        s2 += v.y;
      }
      s1 = group_sum(s1, 32);
      s2 = group_sum(s2, 32);
      if (lane == 0) stat[i] = make_float2(s1 * k.inv_total, s2 * k.inv_total);
    }
  }
  __syncthreads();
  if (MODE == kSlab && k.parts > 1) cluster_arrive();

  // write: gx = du * (gamma rstd) - rstd s1 - xh * (rstd s2)
  if (gx && p.nv > 0) {
    f32x2 c1[NP], c2[NP], c3[NP];
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      const float2 u = stat[gi[2 * e]], v = stat[gi[2 * e + 1]];
      c1[e] = mul_f32x2(ga[e], rs[e]);
      c2[e] = neg(mul_f32x2(pack_f32x2(u.x, v.x), rs[e]));
      c3[e] = neg(mul_f32x2(pack_f32x2(u.y, v.y), rs[e]));
    }
    T* op = gx + first * g.xs + g.xo + p.c;
    auto put = [&](int at) {
      f32x2 xh[NP], du[NP];
      eval(at, xh, du);
#pragma unroll
      for (int e = 0; e < NP; ++e) du[e] = fma2(du[e], c1[e], fma2(xh[e], c3[e], c2[e]));
      L::store(op, k.vpr, p.nv, L::pack(du));
    };
    if constexpr (MODE == kSlab) {
      for (int j = 0; j < mine; ++j, op += xstep) put(at0 + j * dstep);
    } else {
      for (int i = 0; i < batches; ++i) {
        copies_wait<1>();
#pragma unroll
        for (int h = 0; h < kBatch; ++h, op += xstep)
          if (i * kBatch + h < mine) put(slot(i * kBatch + h));
        fetch(i + 2);
      }
    }
  }
  if (MODE == kSlab && k.parts > 1) cluster_wait();
}

// ---- launches --------------------------------------------------------------

// cluster: a slab's blocks; dependent: after the sums of the same call
template <typename... P, typename... A>
cudaError_t launch(void (*kern)(P...), const Norm& g, const Plan& k, bool cluster, bool dependent, int pass,
                   cudaStream_t s, A... args) {
  const int smem = k.data_bytes + scratch_bytes(k, pass);
  if (smem > 48 * 1024) {
    // one limit for every shape: calls from several threads do not lower each other's
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid((unsigned)(g.N * k.slices * k.parts));
  if (dependent) return launch_dependent(kern, grid, dim3(kNT), (size_t)smem, s, args...);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)k.parts;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kNT);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = cluster ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int V, bool STR>
cudaError_t fwd_of(const Norm& g, const Plan& k, bool slab, const T* x, const T* gamma, const T* beta, T* y, float* mean,
                   float* rstd, const Act8& x8, const Sums& sums, cudaStream_t s) {
  const int keep = x8.codes ? x8.src : kSrcFull;
  auto one = [&](auto kern, bool cluster, bool dependent) {
    return launch(kern, g, k, cluster, dependent, 0, s, g, k, x, gamma, beta, y, mean, rstd, x8, sums.groups);
  };
  cudaError_t e = cudaErrorInvalidValue;
#define X(KEEP)                                                              \
  if (keep == KEEP) e = slab ? one(fwd_kernel<T, V, STR, KEEP, kSlab>, true, false) \
                             : one(fwd_kernel<T, V, STR, KEEP, kSums>, false, false);
  X(kSrcFull)
  if constexpr (!STR) {
    X(kSrcI8) X(kSrcE4M3)
  }
#undef X
  if (slab || e != cudaSuccess) return e;
  return one(fwd_kernel<T, V, STR, kSrcFull, kApply>, false, true);
}

template <typename T, int V, bool STR>
cudaError_t bwd_of(const Norm& g, const Plan& k, bool slab, const T* x, const Act8& x8, const T* gy, const T* gamma,
                   const T* beta, const float* mean, const float* rstd, T* gx, const Sums& sums, cudaStream_t s) {
  const int src = x ? kSrcFull : x8.src;
  auto one = [&](auto kern, bool cluster, bool dependent) {
    return launch(kern, g, k, cluster, dependent, 1, s, g, k, x, x8, gy, gamma, beta, mean, rstd, gx, sums);
  };
#define X(SRC)                                                               \
  if (src == SRC) {                                                          \
    if (slab) return one(bwd_kernel<T, V, STR, SRC, kSlab>, true, false);           \
    const cudaError_t e = one(bwd_kernel<T, V, STR, SRC, kSums>, false, false);     \
    return e != cudaSuccess || !gx ? e : one(bwd_kernel<T, V, STR, SRC, kApply>, false, true); \
  }
  X(kSrcFull) X(kSrcI8) X(kSrcE4M3)
#undef X
  return cudaErrorInvalidValue;
}

#define DW_SLAB_LAYOUTS(X)                                    \
  if (k.strided) { X(4, true) }                               \
  if constexpr (sizeof(T) == 2) {                             \
    if (k.V == 8) { X(8, false) }                             \
  }                                                           \
  if (k.V == 4) { X(4, false) }

template <typename T>
cudaError_t run_fwd(const Norm& g, const Plan& k, bool slab, const T* x, const T* gamma, const T* beta, T* y,
                    float* mean, float* rstd, const Act8& x8, const Sums& sums, cudaStream_t s) {
#define X(V, STR) return fwd_of<T, V, STR>(g, k, slab, x, gamma, beta, y, mean, rstd, x8, sums, s);
  DW_SLAB_LAYOUTS(X)
#undef X
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t run_bwd(const Norm& g, const Plan& k, bool slab, const T* x, const Act8& x8, const T* gy, const T* gamma,
                    const T* beta, const float* mean, const float* rstd, T* gx, const Sums& sums, cudaStream_t s) {
#define X(V, STR) return bwd_of<T, V, STR>(g, k, slab, x, x8, gy, gamma, beta, mean, rstd, gx, sums, s);
  DW_SLAB_LAYOUTS(X)
#undef X
  return cudaErrorInvalidValue;
}

}  // namespace slab
}  // namespace norm
}  // namespace dwconv
