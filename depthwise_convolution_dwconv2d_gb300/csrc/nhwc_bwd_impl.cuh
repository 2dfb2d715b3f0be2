// Channels-last depthwise backward: the row-walking kernels.
//
// In this layout a channel's filter is a lane's own, so gx and gw need no
// matrix product and no exchange between lanes: a thread owns two channels
// (the two lanes of fma.rn.f32x2) and a strip of PX columns, walks down the
// rows of its band, and keeps the filter and the filter gradient in
// registers. With u = i + ph and v = j + pw for the input position (i, j),
//
//   gx[u, v]  = sum_{a, b} w[a, b] gy[(u - a) / S, (v - b) / S]
//   gw[a, b] += x[u, v] gy[(u - a) / S, (v - b) / S]
//
// over the a, b that divide: both read the same window of gy, so one pass
// over gy serves both. gb takes each gy once, through the tap at the
// filter's centre: a padding of at most (K - 1) / 2 makes its position an
// input position for every output.
//
// A warp reads and writes 64 channels of a pixel, one 128-byte line in 16
// bits. Neighbouring strips sit in neighbouring warps of a block, so the
// columns that windows share come from L1.
//
// Blocks keep one tile of channels for all of their items (sample, band of
// rows, strip), so the filter gradient leaves registers once per block: its
// row lanes are joined in shared memory in lane order, and a second launch
// adds the blocks' sums in block order.
#pragma once

#include <type_traits>

#include "nhwc_bwd.h"
#include "vec.cuh"

namespace dwconv {
namespace nhwc {
namespace walk {

// ---- pairs of channels -----------------------------------------------------

// Two channels as loaded: 32 bits of the storage type, two floats, or two
// codes with their block's scale.
template <typename T, int SRC> struct Raw { uint32_t v; };
template <> struct Raw<float, kSrcFull> { f32x2 v; };
template <typename T> struct Raw<T, kSrcI8> { uint32_t v; float s; };
template <typename T> struct Raw<T, kSrcE4M3> { uint32_t v; float s; };

template <typename T, int SRC>
__device__ __forceinline__ Raw<T, SRC> zero_raw() { return Raw<T, SRC>{}; }

// PAIR: the two channels are one aligned access; otherwise `two` says whether
// the second exists.
template <typename T, bool PAIR>
__device__ __forceinline__ Raw<T, kSrcFull> load_pair(const T* p, bool two) {
  Raw<T, kSrcFull> r;
  if constexpr (sizeof(T) == 4) {
    if constexpr (PAIR) {
      const float2 f = __ldg(reinterpret_cast<const float2*>(p));
      r.v = pack_f32x2(f.x, f.y);
    } else {
      r.v = pack_f32x2(__ldg(p), two ? __ldg(p + 1) : 0.f);
    }
  } else {
    if constexpr (PAIR) {
      r.v = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else {
      const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
      r.v = (uint32_t)__ldg(h) | (two ? (uint32_t)__ldg(h + 1) << 16 : 0u);
    }
  }
  return r;
}

template <typename T, int SRC, bool PAIR>
__device__ __forceinline__ Raw<T, SRC> load_code_pair(const Act8& t, int64_t row, int64_t C, int ch, bool two) {
  Raw<T, SRC> r;
  const uint8_t* p = t.codes + row * C + ch;
  if constexpr (PAIR) {
    r.v = __ldg(reinterpret_cast<const unsigned short*>(p));
  } else {
    r.v = (uint32_t)__ldg(p) | (two ? (uint32_t)__ldg(p + 1) << 8 : 0u);
  }
  r.s = __ldg(t.scales + row * t.nblk + (ch >> t.shift));  // ch is even: both channels are of one block
  return r;
}

template <typename T, int SRC>
__device__ __forceinline__ f32x2 widen(const Raw<T, SRC>& r) {
  if constexpr (SRC == kSrcI8) {
    const uint32_t u = r.v ^ 0x8080u;
    const float a = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7650)) - 8388736.0f;
    const float b = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7651)) - 8388736.0f;
    return pack_f32x2(__fmul_rn(a, r.s), __fmul_rn(b, r.s));
  } else if constexpr (SRC == kSrcE4M3) {
    float a, b;
    e4m3_pair((uint16_t)r.v, a, b);
    return pack_f32x2(__fmul_rn(a, r.s), __fmul_rn(b, r.s));
  } else if constexpr (sizeof(T) == 4) {
    return r.v;
  } else if constexpr (std::is_same<T, __half>::value) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.v));
    return pack_f32x2(f.x, f.y);
  } else {
    return pack_f32x2(__uint_as_float(r.v << 16), __uint_as_float(r.v & 0xffff0000u));
  }
}

template <typename T, bool PAIR>
__device__ __forceinline__ void store_pair(T* p, f32x2 v, bool two, bool accumulate) {
  float a, b;
  unpack_f32x2(v, a, b);
  if (accumulate) {
    a += to_f<T>(p[0]);
    if (PAIR || two) b += to_f<T>(p[1]);
  }
  if constexpr (PAIR && sizeof(T) == 4) {
    *reinterpret_cast<float2*>(p) = make_float2(a, b);
  } else if constexpr (PAIR) {
    T h[2] = {from_f<T>(a), from_f<T>(b)};
    *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<const uint32_t*>(h);
  } else {
    p[0] = from_f<T>(a);
    if (two) p[1] = from_f<T>(b);
  }
}

// ---- items -----------------------------------------------------------------

// Sums the block's NACC pairs per thread over its row lanes, in lane order,
// into ws[chunk][tap][channel].
template <int NT, int NACC>
__device__ __forceinline__ void join_lanes(const Geom& g, const f32x2* acc, int C, int ch, int chunk, float* ws) {
  constexpr int kAt = 5;  // taps joined at a time
  __shared__ f32x2 sm[kAt * NT];
  const int ct = 1 << g.ct_log, lanes = NT >> g.ct_log;
#pragma unroll
  for (int k = 0; k < NACC; k += kAt) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kAt; ++q)
      if (k + q < NACC) sm[q * NT + threadIdx.x] = acc[k + q];
    __syncthreads();
    for (int i = threadIdx.x; i < kAt * ct; i += NT) {
      const int q = i >> g.ct_log, l = i & (ct - 1);
      if (k + q >= NACC) break;
      float a = 0.f, b = 0.f;
      for (int r = 0; r < lanes; ++r) {
        float u, v;
        unpack_f32x2(sm[q * NT + r * ct + l], u, v);
        a += u;
        b += v;
      }
      const int c = ch + 2 * l;
      float* o = ws + ((int64_t)chunk * NACC + k + q) * C + c;
      if (c < C) o[0] = a;
      if (c + 1 < C) o[1] = b;
    }
  }
}

// 3x3 filters: gx, gw and gb in one walk. The gy rows of the last steps stay
// in registers (a ring whose slots the unrolled loop names), so each gy and
// each x of the strip is loaded once; the next step's loads are issued before
// this step's arithmetic.
template <typename T, int SRC, int S, bool PAIR>
__global__ void __launch_bounds__(256, 2)
ring3_kernel(Conv c, Geom g, const T* __restrict__ x, Act8 x8, const T* __restrict__ gy, const T* __restrict__ w,
             T* __restrict__ gx, float* __restrict__ ws) {
  constexpr int NT = 256, K = 3, PX = 4;
  constexpr int D = (K - 1) / S, RD = D + 1, WIN = D + (PX - 1) / S + 1;
  const int ct = 1 << g.ct_log;
  const int tile = blockIdx.x % g.tiles, chunk = blockIdx.x / g.tiles;
  const int ch0 = tile * 2 * ct;
  const int ch = ch0 + 2 * (int)(threadIdx.x & (ct - 1));
  const int lane = threadIdx.x >> g.ct_log, lanes = NT >> g.ct_log;
  const int C = (int)c.C, H = (int)c.H, W = (int)c.W, Ho = (int)c.Ho, Wo = (int)c.Wo;
  const bool on = ch < C, two = ch + 1 < C;

  f32x2 wr[K * K], acc[K * K + 1];
#pragma unroll
  for (int k = 0; k < K * K; ++k) {
    wr[k] = 0;
    if (on && g.want_gx)
      wr[k] = pack_f32x2(ld(w + (int64_t)ch * K * K + k), two ? ld(w + (int64_t)(ch + 1) * K * K + k) : 0.f);
  }
#pragma unroll
  for (int k = 0; k <= K * K; ++k) acc[k] = 0;

  for (int64_t grp = chunk; grp < g.groups; grp += g.chunks) {
    const int64_t item = grp * lanes + lane;
    if (item >= g.items || !on) continue;
    const int strip = (int)(item % g.strips);
    const int64_t q = item / g.strips;
    const int64_t n = q / g.bands;
    const int tb = g.t_begin + (int)(q - n * g.bands) * g.band;
    const int te = min(tb + g.band, g.t_end);
    const int v0 = g.v_begin + strip * PX;
    const int ow0 = v0 / S - D, iw0 = v0 - c.pw;
    uint32_t wok = 0, xok = 0;  // columns inside gy / x
#pragma unroll
    for (int j = 0; j < WIN; ++j) wok |= (ow0 + j >= 0 && ow0 + j < Wo) ? 1u << j : 0u;
#pragma unroll
    for (int p = 0; p < PX; ++p) xok |= (iw0 + p >= 0 && iw0 + p < W) ? 1u << p : 0u;
    const T* gyn = gy + ((n * Ho) * Wo + ow0) * c.ctot + c.off + ch;
    const int64_t xrow = n * H * (int64_t)W + iw0;

    Raw<T, kSrcFull> rg[WIN];
    Raw<T, SRC> rx[S * PX];
    auto fetch_gy = [&](int t) {
#pragma unroll
      for (int j = 0; j < WIN; ++j) {
        rg[j] = zero_raw<T, kSrcFull>();
        if (t >= 0 && t < Ho && ((wok >> j) & 1))
          rg[j] = load_pair<T, PAIR>(gyn + ((int64_t)t * Wo + j) * c.ctot, two);
      }
    };
    auto fetch_x = [&](int t) {
#pragma unroll
      for (int r = 0; r < S; ++r) {
        const int ih = S * t + r - c.ph;
#pragma unroll
        for (int p = 0; p < PX; ++p) {
          rx[r * PX + p] = zero_raw<T, SRC>();
          if (g.want_gw && ih >= 0 && ih < H && ((xok >> p) & 1)) {
            const int64_t row = xrow + (int64_t)ih * W + p;
            if constexpr (SRC == kSrcFull) {
              if (x) rx[r * PX + p] = load_pair<T, PAIR>(x + row * C + ch, two);
            } else {
              rx[r * PX + p] = load_code_pair<T, SRC, PAIR>(x8, row, C, ch, two);
            }
          }
        }
      }
    };

    f32x2 ring[RD][WIN];
#pragma unroll
    for (int d = 1; d <= D; ++d) {  // step tb is phase 0: row tb - d in slot (0 - d) mod RD
      fetch_gy(tb - d);
#pragma unroll
      for (int j = 0; j < WIN; ++j) ring[RD - d][j] = widen<T, kSrcFull>(rg[j]);
    }
    fetch_gy(tb);
    fetch_x(tb);
    for (int t = tb; t < te;) {
#pragma unroll
      for (int i = 0; i < RD; ++i) {
        if (t >= te) break;
        f32x2 xv[S * PX];
#pragma unroll
        for (int j = 0; j < WIN; ++j) ring[i][j] = widen<T, kSrcFull>(rg[j]);
#pragma unroll
        for (int p = 0; p < S * PX; ++p) xv[p] = widen<T, SRC>(rx[p]);
        if (t + 1 < te) {
          fetch_gy(t + 1);
          fetch_x(t + 1);
        }
#pragma unroll
        for (int r = 0; r < S; ++r) {
          f32x2 out[PX];
#pragma unroll
          for (int p = 0; p < PX; ++p) out[p] = 0;
#pragma unroll
          for (int a = r; a < K; a += S) {
            const int slot = (i - (a - r) / S + RD) % RD;
#pragma unroll
            for (int p = 0; p < PX; ++p)
#pragma unroll
              for (int b = 0; b < K; ++b) {
                if ((p - b) % S != 0) continue;
                const f32x2 gv = ring[slot][D + (p - b) / S];
                fma_f32x2(out[p], wr[a * K + b], gv);
                fma_f32x2(acc[a * K + b], xv[r * PX + p], gv);
                if (a == K / 2 && b == K / 2) fma_f32x2(acc[K * K], pack_f32x2(1.f, 1.f), gv);
              }
          }
          const int ih = S * t + r - c.ph;
          if (g.want_gx && ih >= 0 && ih < H) {
            T* o = gx + (xrow + (int64_t)ih * W) * C + ch;
#pragma unroll
            for (int p = 0; p < PX; ++p)
              if ((xok >> p) & 1) store_pair<T, PAIR>(o + (int64_t)p * C, out[p], two, g.accumulate);
          }
        }
        ++t;
      }
    }
  }
  if (g.want_gw) join_lanes<NT, K * K + 1>(g, acc, C, ch0, chunk, ws);
}

// 5x5 and 7x7 filters: gx (GW = false) or gw and gb (GW = true), whose filter
// or gradient alone takes up to 98 registers. A step owns RY = 2 rows of the
// strip and reads each row of gy that they meet once (from L1 after the
// first step that meets it), for up to 2 K^2 PX products.
template <typename T, int SRC, int K, int S, bool GW, bool PAIR>
__global__ void __launch_bounds__(128, 3)
block_kernel(Conv c, Geom g, const T* __restrict__ x, Act8 x8, const T* __restrict__ gy, const T* __restrict__ w,
             T* __restrict__ gx, float* __restrict__ ws) {
  constexpr int NT = 128, PX = 8, RY = 2, M = RY / S;
  constexpr int D = (K - 1) / S, WIN = D + (PX - 1) / S + 1;
  const int ct = 1 << g.ct_log;
  const int tile = blockIdx.x % g.tiles, chunk = blockIdx.x / g.tiles;
  const int ch0 = tile * 2 * ct;
  const int ch = ch0 + 2 * (int)(threadIdx.x & (ct - 1));
  const int lane = threadIdx.x >> g.ct_log, lanes = NT >> g.ct_log;
  const int C = (int)c.C, H = (int)c.H, W = (int)c.W, Ho = (int)c.Ho, Wo = (int)c.Wo;
  const bool on = ch < C, two = ch + 1 < C;

  f32x2 acc[K * K + (GW ? 1 : 0)];  // the filter, or its gradient and the bias's
#pragma unroll
  for (int k = 0; k < K * K + (GW ? 1 : 0); ++k) {
    acc[k] = 0;
    if (!GW && on)
      acc[k] = pack_f32x2(ld(w + (int64_t)ch * K * K + k), two ? ld(w + (int64_t)(ch + 1) * K * K + k) : 0.f);
  }

  for (int64_t grp = chunk; grp < g.groups; grp += g.chunks) {
    const int64_t item = grp * lanes + lane;
    if (item >= g.items || !on) continue;
    const int strip = (int)(item % g.strips);
    const int64_t q = item / g.strips;
    const int64_t n = q / g.bands;
    const int tb = g.t_begin + (int)(q - n * g.bands) * g.band;
    const int te = min(tb + g.band, g.t_end);
    const int v0 = g.v_begin + strip * PX;
    const int ow0 = v0 / S - D, iw0 = v0 - c.pw;
    uint32_t wok = 0, xok = 0;
#pragma unroll
    for (int j = 0; j < WIN; ++j) wok |= (ow0 + j >= 0 && ow0 + j < Wo) ? 1u << j : 0u;
#pragma unroll
    for (int p = 0; p < PX; ++p) xok |= (iw0 + p >= 0 && iw0 + p < W) ? 1u << p : 0u;
    const T* gyn = gy + ((n * Ho) * Wo + ow0) * c.ctot + c.off + ch;
    const int64_t xrow = n * H * (int64_t)W + iw0;

    for (int t = tb; t < te; t += M) {
      f32x2 own[RY * PX];  // x of the strip, or its gx
#pragma unroll
      for (int r = 0; r < RY; ++r) {
        const int ih = S * t + r - c.ph;
#pragma unroll
        for (int p = 0; p < PX; ++p) {
          own[r * PX + p] = 0;
          if (GW && ih >= 0 && ih < H && ((xok >> p) & 1)) {
            const int64_t row = xrow + (int64_t)ih * W + p;
            if constexpr (SRC == kSrcFull) {
              if (x) own[r * PX + p] = widen<T, SRC>(load_pair<T, PAIR>(x + row * C + ch, two));
            } else {
              own[r * PX + p] = widen<T, SRC>(load_code_pair<T, SRC, PAIR>(x8, row, C, ch, two));
            }
          }
        }
      }
#pragma unroll
      for (int e = -D; e <= (RY - 1) / S; ++e) {  // gy row t + e meets the filter's rows a = r - S e
        f32x2 gv[WIN];
#pragma unroll
        for (int j = 0; j < WIN; ++j) {
          Raw<T, kSrcFull> v = zero_raw<T, kSrcFull>();
          if (t + e >= 0 && t + e < Ho && ((wok >> j) & 1))
            v = load_pair<T, PAIR>(gyn + ((int64_t)(t + e) * Wo + j) * c.ctot, two);
          gv[j] = widen<T, kSrcFull>(v);
        }
#pragma unroll
        for (int r = 0; r < RY; ++r) {
          const int a = r - S * e;
          if (a < 0 || a >= K) continue;
#pragma unroll
          for (int p = 0; p < PX; ++p)
#pragma unroll
            for (int b = 0; b < K; ++b) {
              if ((p - b) % S != 0) continue;
              const f32x2 v = gv[D + (p - b) / S];
              if (GW) {
                fma_f32x2(acc[a * K + b], own[r * PX + p], v);
                if (a == K / 2 && b == K / 2) fma_f32x2(acc[K * K], pack_f32x2(1.f, 1.f), v);
              } else {
                fma_f32x2(own[r * PX + p], acc[a * K + b], v);
              }
            }
        }
      }
      if (!GW) {
#pragma unroll
        for (int r = 0; r < RY; ++r) {
          const int ih = S * t + r - c.ph;
          if (ih < 0 || ih >= H) continue;
          T* o = gx + (xrow + (int64_t)ih * W) * C + ch;
#pragma unroll
          for (int p = 0; p < PX; ++p)
            if ((xok >> p) & 1) store_pair<T, PAIR>(o + (int64_t)p * C, own[r * PX + p], two, g.accumulate);
        }
      }
    }
  }
  if constexpr (GW) join_lanes<NT, K * K + 1>(g, acc, C, ch0, chunk, ws);
}

// ---- launches --------------------------------------------------------------

template <typename T, int SRC, bool PAIR>
cudaError_t launch(const Conv& c, const Geom& g, const T* x, const Act8& x8, const T* gy, const T* w, T* gx, float* ws,
                   cudaStream_t s) {
  const unsigned grid = (unsigned)(g.tiles * g.chunks);
  if (c.kh == 3) {
    if (c.sh == 1)
      ring3_kernel<T, SRC, 1, PAIR><<<grid, 256, 0, s>>>(c, g, x, x8, gy, w, gx, ws);
    else
      ring3_kernel<T, SRC, 2, PAIR><<<grid, 256, 0, s>>>(c, g, x, x8, gy, w, gx, ws);
    return cudaGetLastError();
  }
#define X(K, S)                                                                                       \
  if (c.kh == K && c.sh == S) {                                                                       \
    if (g.want_gx) block_kernel<T, kSrcFull, K, S, false, PAIR><<<grid, 128, 0, s>>>(c, g, x, x8, gy, w, gx, ws); \
    if (g.want_gw) block_kernel<T, SRC, K, S, true, PAIR><<<grid, 128, 0, s>>>(c, g, x, x8, gy, w, gx, ws);       \
  }
  X(5, 1) X(5, 2) X(7, 1) X(7, 2)
#undef X
  return cudaGetLastError();
}

template <typename T>
cudaError_t run(const Conv& c, const Geom& g, bool pair, const T* x, const Act8& x8, const T* gy, const T* w, T* gx,
                float* ws, cudaStream_t s) {
  const int src = x || !x8.codes ? kSrcFull : x8.src;
#define X(SRC)                                                              \
  if (src == SRC)                                                           \
    return pair ? launch<T, SRC, true>(c, g, x, x8, gy, w, gx, ws, s)       \
                : launch<T, SRC, false>(c, g, x, x8, gy, w, gx, ws, s);
  X(kSrcFull) X(kSrcI8) X(kSrcE4M3)
#undef X
  return cudaErrorInvalidValue;
}

}  // namespace walk
}  // namespace nhwc
}  // namespace dwconv
