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

#include "dependent.cuh"
#include "nhwc_bwd.h"
#include "tma.cuh"
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
    const f32x2 m = pack_f32x2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7650)),
                               __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7651)));
    return mul_f32x2(add_f32x2(m, pack_f32x2(-8388736.0f, -8388736.0f)), pack_f32x2(r.s, r.s));
  } else if constexpr (SRC == kSrcE4M3) {
    float a, b;
    e4m3_pair((uint16_t)r.v, a, b);
    return mul_f32x2(pack_f32x2(a, b), pack_f32x2(r.s, r.s));
  } else if constexpr (sizeof(T) == 4) {
    return r.v;
  } else if constexpr (std::is_same<T, __half>::value) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.v));
    return pack_f32x2(f.x, f.y);
  } else {
    return pack_f32x2(__uint_as_float(r.v << 16), __uint_as_float(r.v & 0xffff0000u));
  }
}

// two aligned channels, each rounded once
__device__ __forceinline__ void put_pair(float* p, float a, float b) { *reinterpret_cast<float2*>(p) = make_float2(a, b); }
__device__ __forceinline__ void put_pair(__half* p, float a, float b) {
  *reinterpret_cast<__half2*>(p) = __floats2half2_rn(a, b);
}
__device__ __forceinline__ void put_pair(__nv_bfloat16* p, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}

template <typename T, bool PAIR>
__device__ __forceinline__ void store_pair(T* p, f32x2 v, bool two, bool accumulate) {
  float a, b;
  unpack_f32x2(v, a, b);
  if (accumulate) {
    a += to_f<T>(p[0]);
    if (PAIR || two) b += to_f<T>(p[1]);
  }
  if constexpr (PAIR) {
    put_pair(p, a, b);
  } else {
    p[0] = from_f<T>(a);
    if (two) p[1] = from_f<T>(b);
  }
}

// Stores a strip of PX pixels, C channels apart: with no branch per pixel
// where all of it is inside and nothing is added to.
template <typename T, bool PAIR, int PX>
__device__ __forceinline__ void store_strip(T* o, int64_t C, const f32x2* v, uint32_t ok, bool two, bool accumulate) {
  if (PAIR && ok == (1u << PX) - 1 && !accumulate) {
#pragma unroll
    for (int p = 0; p < PX; ++p) {
      float a, b;
      unpack_f32x2(v[p], a, b);
      put_pair(o + p * C, a, b);
    }
  } else {
#pragma unroll
    for (int p = 0; p < PX; ++p)
      if ((ok >> p) & 1) store_pair<T, PAIR>(o + p * C, v[p], two, accumulate);
  }
}

// Loads from a 32-bit shared address: a register and a constant make one
// instruction. Volatile, to stay behind the wait for the copy that wrote it.
__device__ __forceinline__ uint32_t lds_u16(uint32_t at) {
  unsigned short v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
template <typename T>
__device__ __forceinline__ Raw<T, kSrcFull> lds_pair(uint32_t at) {
  Raw<T, kSrcFull> r;
  if constexpr (sizeof(T) == 4) {
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(r.v) : "r"(at));
  } else {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r.v) : "r"(at));
  }
  return r;
}

// ---- items -----------------------------------------------------------------

// Sums the block's NACC pairs per thread over its row lanes, in lane order,
// into ws[chunk][tap][channel]. NT: the most threads of a block.
template <int NT, int NACC>
__device__ __forceinline__ void join_lanes(int ct_log, const f32x2* acc, int C, int ch, int chunk, float* ws) {
  constexpr int kAt = 5;  // taps joined at a time
  __shared__ f32x2 sm[kAt * NT];
  const int ct = 1 << ct_log, lanes = blockDim.x >> ct_log;
#pragma unroll
  for (int k = 0; k < NACC; k += kAt) {
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kAt; ++q)
      if (k + q < NACC) sm[q * NT + threadIdx.x] = acc[k + q];
    __syncthreads();
    for (int i = threadIdx.x; i < kAt * ct; i += blockDim.x) {
      const int q = i >> ct_log, l = i & (ct - 1);
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

// 3x3 filters with plain loads: gx, gw and gb in one walk. The gy rows of the
// last steps stay in registers (a ring whose slots the unrolled loop names),
// so each gy and each x of the strip is loaded once; the next step's loads
// are issued before this step's arithmetic. It serves what the staged kernel
// does not: fewer than 24 channels, pointers off 16 bytes. Masks, addresses
// and scales make six instructions of every product: 77 us at 64x56x56x128
// bf16 from integer codes (1.7 TB/s), where the staged kernel takes 41. At
// stride 1 the fp32 forms spill 212 to 296 bytes of a thread.
template <typename T, int SRC, int S, bool PAIR>
__global__ void __launch_bounds__(kRingThreads, kRingBlocks)
ring3_kernel(Conv c, Geom g, const T* __restrict__ x, Act8 x8, const T* __restrict__ gy, const T* __restrict__ w,
             T* __restrict__ gx, float* __restrict__ ws) {
  constexpr int NT = kRingThreads, K = 3, PX = 4;
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
            store_strip<T, PAIR, PX>(gx + (xrow + (int64_t)ih * W) * C + ch, C, out, xok, two, g.accumulate);
          }
        }
        ++t;
      }
    }
  }
  if (g.want_gw) join_lanes<NT, K * K + 1>(g.ct_log, acc, C, ch0, chunk, ws);
}

// 3x3 filters, staged: the same walk with the rows of gy and x brought to
// shared memory by the tensor memory accelerator, some stages ahead. The
// copies' zero fill outside the tensors is the padding, so the loop has no
// column masks. A stage is as many rows as the ring has slots: row i of a
// stage is slot i, and a stage costs one barrier and one wait. All lanes of a
// block walk the same rows.
//
// Bound by latency with 14 warps an SM: 64x56x56x128 bf16 from integer codes
// takes 41 us (3.2 TB/s of the floor's bytes, 0.48 of the measured copy; 22.6
// TFLOP/s), issue active 55 % of the time, fixed waits the first stall (27 %),
// for 24.9 M warp instructions, about 190 for the 78 packed products of a row of four
// pixels (unpacking, decoding, stores and the item's start are the rest);
// fp32 at 128 samples, with nothing to unpack, runs at 5.9 TB/s, at the
// memory. Four blocks of four warps per SM at up to 128 registers: two of
// seven warps took 55 us (fewer warps, coarser items), five at 96 registers
// spill (68 us for the call against 54).
template <typename T, int SRC, int S, int CT>
__global__ void __launch_bounds__(kStagedThreads, kStagedBlocks)
staged3_kernel(Conv c, Staged g, const __grid_constant__ CUtensorMap map_gy, const __grid_constant__ CUtensorMap map_x,
               Act8 x8, unsigned int* timeouts, const T* __restrict__ w, T* __restrict__ gx, float* __restrict__ ws) {
  constexpr int K = 3, PX = 4, NT = kStagedThreads;
  constexpr int D = (K - 1) / S, RD = D + 1, WIN = D + (PX - 1) / S + 1;
  constexpr bool kCode = SRC != kSrcFull;
  constexpr int GP = 2 * CT * (int)sizeof(T);             // bytes of a staged pixel of gy
  constexpr int XP = kCode ? 2 * CT : GP;                 // of x
  extern __shared__ __align__(16) unsigned char smdyn[];
  __shared__ __align__(8) uint64_t full[kMaxStages];
  dependents_may_start();
  const int base = (int)((128 - (tma::smem_u32(smdyn) & 127)) & 127);
  const uint32_t sm0 = tma::smem_u32(smdyn) + base;
  const int tile = blockIdx.x % g.tiles, chunk = blockIdx.x / g.tiles;
  const int ch0 = tile * 2 * CT;
  const int pl = threadIdx.x & (CT - 1);
  const int ch = ch0 + 2 * pl;
  const int lane = threadIdx.x / CT;
  const int ls = lane % g.cs, ln = lane / g.cs;           // strip and sample of the lane
  const int la = min(ln, g.ns - 1);                       // a lane past the last sample reads within the stage
  const int C = (int)c.C, W = (int)c.W;
  const bool two = ch + 1 < C;
  const uint32_t g_at = sm0 + (la * RD * g.gc + ls * (PX / S)) * GP + pl * (GP / CT);
  const uint32_t x_at = sm0 + g.x_at + (la * RD * S * g.xc + ls * PX) * XP + pl * (XP / CT);

  // What a row needs besides its data goes through shared memory, so that it stays in registers: from the kernel's
  // parameters the compiler recomputes it in every row (50 integer instructions and 13 parameter loads a row).
  __shared__ uint32_t keep[8];
  if (threadIdx.x == 0) {
    for (int i = 0; i < g.stages; ++i) tma::mbar_init(&full[i], 1);
    tma::fence_init();
    const uint64_t row = (uint64_t)c.W * c.C * sizeof(T);
    keep[0] = g.gc * GP;
    keep[1] = g.xc * XP;
    keep[2] = (uint32_t)(c.C * sizeof(T));
    keep[3] = (uint32_t)row;
    keep[4] = (uint32_t)(row >> 32);
    keep[5] = (uint32_t)c.H;
    keep[6] = (uint32_t)c.ph;
    keep[7] = (uint32_t)(c.W * x8.nblk * 4);
  }
  __syncthreads();
  const uint32_t keep0 = tma::smem_u32(keep);
  const uint32_t grow = lds_u32(keep0), xrow = lds_u32(keep0 + 4);    // bytes of a staged row of gy, of x
  const uint32_t pixel = lds_u32(keep0 + 8);                          // bytes of a pixel and a row of gx
  const uint64_t row = lds_u32(keep0 + 12) | (uint64_t)lds_u32(keep0 + 16) << 32;
  const int H = (int)lds_u32(keep0 + 20), ph = (int)lds_u32(keep0 + 24);
  const uint32_t srow = lds_u32(keep0 + 28);                          // bytes of a row of scales

  struct Item {
    int n0, v0, tb, te;  // first sample and column of the block, rows of the band
  };
  auto item_of = [&](int i) {
    Item it;
    uint32_t q, n;
    const uint32_t seg = g.d_segs.divmod((uint32_t)i, q);
    const uint32_t band = g.d_bands.divmod(q, n);
    it.n0 = (int)n * g.ns;
    it.v0 = g.v_begin + (int)seg * g.cs * PX;
    it.tb = g.t_begin + (int)band * g.band;
    it.te = min(it.tb + g.band, g.t_end);
    return it;
  };

  // the next copy to issue (thread 0): gy rows p_t .. p_t + RD - 1 of item p_item
  int p_item = chunk, p_slot = 0;
  Item p_it = item_of(p_item);
  int p_t = p_it.tb - D;
  auto issue = [&]() {
    if (p_item >= g.items) return;
    unsigned char* const slot = smdyn + base + p_slot * g.stage_bytes;
    tma::fence_async_smem();
    tma::mbar_expect_tx(&full[p_slot], (uint32_t)(g.gy_bytes + (g.want_x ? g.x_bytes : 0)));
    tma::load_4d(slot, &map_gy, ch0, p_it.v0 / S - D, p_t, p_it.n0, &full[p_slot]);
    if (g.want_x)
      tma::load_4d(slot + g.x_at, &map_x, kCode ? ch0 / 2 : ch0, p_it.v0 - c.pw, p_t * S - c.ph, p_it.n0, &full[p_slot]);
    p_slot = p_slot + 1 == g.stages ? 0 : p_slot + 1;
    p_t += RD;
    if (p_t >= p_it.te) {
      p_item += g.chunks;
      p_it = item_of(p_item);
      p_t = p_it.tb - D;
    }
  };
  wait_for_previous();  // the aligned copies of the same call, where there are any
  if (threadIdx.x == 0)
    for (int i = 0; i < g.stages - 1; ++i) issue();

  f32x2 wr[K * K], acc[K * K + 1];
#pragma unroll
  for (int k = 0; k < K * K; ++k) {
    wr[k] = 0;
    if (ch < C && g.want_gx)
      wr[k] = pack_f32x2(ld(w + (int64_t)ch * K * K + k), two ? ld(w + (int64_t)(ch + 1) * K * K + k) : 0.f);
  }
#pragma unroll
  for (int k = 0; k <= K * K; ++k) acc[k] = 0;

  int slot = 0;
  uint32_t parity = 0;
  bool first = true;
  for (int item = chunk; item < g.items; item += g.chunks) {
    const Item it = item_of(item);
    const int64_t n = it.n0 + ln;
    const int strip = (it.v0 - g.v_begin) / PX + ls;
    const bool here = ln < g.ns && n < c.N && strip < g.strips, on = here && ch < C;
    const int iw0 = it.v0 + ls * PX - c.pw;
    uint32_t xok = 0;
#pragma unroll
    for (int p = 0; p < PX; ++p) xok |= (iw0 + p >= 0 && iw0 + p < W) ? 1u << p : 0u;
    const int64_t at = n * H * (int64_t)W + (int64_t)(S * it.tb - c.ph) * W + iw0;  // pixel of the band's first row
    char* op = reinterpret_cast<char*>(gx + at * C + ch);
    const int stores = !on || !g.want_gx ? 0 : !g.pair_out ? 3 : xok == (1u << PX) - 1 && !g.accumulate ? 1 : 2;
    // a checkpoint's scales: lanes p + 4 b of the strip's lanes read pixel p, block b of the tile's
    const int sl = pl & 7, sb = (ch0 >> x8.shift) + (sl >> 2);
    const bool scaler = kCode && here && g.want_x && pl < 8 && sb < x8.nblk && ((xok >> (sl & 3)) & 1);
    const int from = (int)(threadIdx.x & 31 & ~(CT - 1)) + 4 * ((ch >> x8.shift) - (ch0 >> x8.shift));
    const char* sp = reinterpret_cast<const char*>(x8.scales + (at + (sl & 3)) * x8.nblk + sb);
    float sc[S];
    auto fetch_scales = [&](int t) {  // t = it.tb, it.tb + 1, ...
#pragma unroll
      for (int r = 0; r < S; ++r) {
        const int ih = S * t + r - ph;
        sc[r] = 0.f;
        if (scaler && (S == 1 || (ih >= 0 && ih < H))) sc[r] = __ldg(reinterpret_cast<const float*>(sp));
        sp += srow;
      }
    };
    if (kCode) fetch_scales(it.tb);

    f32x2 ring[RD][WIN];
    for (int t0 = it.tb - D; t0 < it.te; t0 += RD) {
      if (!first) {  // the stage before this one is free once every thread is here
        __syncthreads();
        slot = slot + 1 == g.stages ? 0 : slot + 1;
        parity ^= slot == 0 ? 1u : 0u;
      }
      first = false;
      if (threadIdx.x == 0) issue();
      if (!tma::mbar_wait(&full[slot], parity, timeouts)) {
        // the copy never landed: let those in flight finish (bounded), then stop
        for (int j = 1; j < g.stages; ++j) {
          const int q = (slot + j) % g.stages;
          tma::mbar_wait(&full[q], q > slot ? parity : parity ^ 1u, nullptr);
        }
        return;
      }
      uint32_t gs = g_at + slot * g.stage_bytes, xs = x_at + slot * g.stage_bytes;
#pragma unroll
      for (int i = 0; i < RD; ++i, gs += grow, xs += S * xrow) {
        const int t = t0 + i;
#pragma unroll
        for (int j = 0; j < WIN; ++j) ring[i][j] = widen<T, kSrcFull>(lds_pair<T>(gs + j * GP));
        if (t < it.tb || t >= it.te) continue;
        f32x2 xv[S * PX];
#pragma unroll
        for (int r = 0; r < S; ++r) {
          const uint32_t q = xs + r * xrow;
#pragma unroll
          for (int p = 0; p < PX; ++p) {
            if constexpr (kCode) {
              Raw<T, SRC> v;
              v.s = __shfl_sync(0xffffffffu, sc[r], from + p);
              v.v = lds_u16(q + p * XP);
              xv[r * PX + p] = widen<T, SRC>(v);
            } else {
              xv[r * PX + p] = widen<T, SRC>(lds_pair<T>(q + p * XP));
            }
          }
        }
        if (kCode) {
          if (t + 1 < it.te) fetch_scales(t + 1);
        }
        if (on) {
#pragma unroll
          for (int r = 0; r < S; ++r) {
            f32x2 out[PX];
#pragma unroll
            for (int a = r; a < K; a += S) {
              const int rs = (i - (a - r) / S + RD) % RD;
#pragma unroll
              for (int b = 0; b < K; ++b)
#pragma unroll
                for (int p = 0; p < PX; ++p) {
                  if ((p - b) % S != 0) continue;
                  const f32x2 gv = ring[rs][D + (p - b) / S];
                  if (a == r && b == p % S) out[p] = mul_f32x2(wr[a * K + b], gv);
                  else fma_f32x2(out[p], wr[a * K + b], gv);
                  fma_f32x2(acc[a * K + b], xv[r * PX + p], gv);
                  if (a == K / 2 && b == K / 2) acc[K * K] = add_f32x2(acc[K * K], gv);
                }
            }
            const int ih = S * t + r - ph;
            if (S == 1 || (ih >= 0 && ih < H)) {  // at stride 1 every owned row is inside
              if (stores == 1) {
                char* o = op;
#pragma unroll
                for (int p = 0; p < PX; ++p, o += pixel) {
                  float a, b;
                  unpack_f32x2(out[p], a, b);
                  put_pair(reinterpret_cast<T*>(o), a, b);
                }
              } else if (stores == 2) {
#pragma unroll
                for (int p = 0; p < PX; ++p)
                  if ((xok >> p) & 1) store_pair<T, true>(reinterpret_cast<T*>(op + p * pixel), out[p], true, g.accumulate);
              } else if (stores == 3) {
#pragma unroll
                for (int p = 0; p < PX; ++p)
                  if ((xok >> p) & 1) store_pair<T, false>(reinterpret_cast<T*>(op + p * pixel), out[p], two, g.accumulate);
              }
            }
            op += row;
          }
        } else {
          op += S * row;
        }
      }
    }
  }
  if (g.want_gw) join_lanes<NT, K * K + 1>(g.ct_log, acc, C, ch0, chunk, ws);
}

// 5x5 and 7x7 filters: gx (GW = false) or gw and gb (GW = true), whose filter
// or gradient alone takes up to 98 registers; both in one launch, each by its
// own blocks. A step owns RY = 2 rows of the strip and reads each row of gy
// that they meet once (from L1 after the first step that meets it), for up to
// 2 K^2 PX products. Plain loads, for what the staged tiles do not serve: two
// blocks per SM, since at three (168 registers) the 7x7 gradient spills (74
// us against 51 at 5x45x51x96 fp32); at two, 7x7 at stride 1 spills 92 to 108
// bytes in bf16, 20 in fp32.
template <typename T, int SRC, int K, int S, bool GW, bool PAIR>
__device__ __forceinline__ void block_walk(const Conv& c, const Geom& g, const T* __restrict__ x, const Act8& x8,
                                           const T* __restrict__ gy, const T* __restrict__ w, T* __restrict__ gx,
                                           float* __restrict__ ws) {
  constexpr int NT = kBlockThreads, PX = 8, RY = 2, M = RY / S;
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
          store_strip<T, PAIR, PX>(gx + (xrow + (int64_t)ih * W) * C + ch, C, own + r * PX, xok, two, g.accumulate);
        }
      }
    }
  }
  if constexpr (GW) join_lanes<NT, K * K + 1>(g.ct_log, acc, C, ch0, chunk, ws);
}

template <typename T, int SRC, int K, int S, bool PAIR>
__global__ void __launch_bounds__(kBlockThreads, kBlockBlocks)
block_kernel(Conv c, Geom g, const T* __restrict__ x, Act8 x8, const T* __restrict__ gy, const T* __restrict__ w,
             T* __restrict__ gx, float* __restrict__ ws) {
  if (g.want_gw && blockIdx.y == 0)
    block_walk<T, SRC, K, S, true, PAIR>(c, g, x, x8, gy, w, gx, ws);
  else
    block_walk<T, kSrcFull, K, S, false, PAIR>(c, g, x, x8, gy, w, gx, ws);
}

// 5x5 and 7x7 filters, staged: a stage is an item, `band` rows of gy with the
// K - 1 above them (a few steps' worth), brought by one copy, and the rows of
// x that they meet by another. gx and gw are separate blocks, as in
// block_kernel; each reads a row of gy for every filter row that meets it,
// from shared memory at constant offsets.
//
// 32x28x28x128 bf16: 33 us for the call at 7x7 (19 TFLOP/s), 19 at 5x5 (17),
// against 99 and 36 with plain loads. The packed products bound it (about 52
// TFLOP/s where all three operands change); on small layers the cold
// instruction cache does: a step is some 400 products of straight code, and a
// block of 5x45x51x96 fp32 7x7 (17 us) takes only a few. With strips of eight
// columns, 800 products, it took 22 us and lost four of every six issue slots.
template <typename T, int SRC, int K, int S, int CT, bool GW>
__device__ __forceinline__ void tile_walk(const Conv& c, const Staged& g, const CUtensorMap* map_gy,
                                          const CUtensorMap* map_x, const Act8& x8, unsigned int* timeouts,
                                          const T* __restrict__ w, T* __restrict__ gx, float* __restrict__ ws) {
  constexpr int PX = tile_px(K), RY = 2, M = RY / S, NT = kTileThreads;
  constexpr int D = (K - 1) / S, WIN = D + (PX - 1) / S + 1;
  constexpr bool kCode = GW && SRC != kSrcFull;
  constexpr int GP = 2 * CT * (int)sizeof(T), XP = kCode ? 2 * CT : GP;
  extern __shared__ __align__(16) unsigned char smdyn[];
  __shared__ __align__(8) uint64_t full[kMaxStages];
  dependents_may_start();
  const int base = (int)((128 - (tma::smem_u32(smdyn) & 127)) & 127);
  const uint32_t sm0 = tma::smem_u32(smdyn) + base;
  const int tile = blockIdx.x % g.tiles, chunk = blockIdx.x / g.tiles;
  const int ch0 = tile * 2 * CT;
  const int pl = threadIdx.x & (CT - 1), ch = ch0 + 2 * pl;
  const int lane = threadIdx.x / CT, ls = lane % g.cs, ln = lane / g.cs, la = min(ln, g.ns - 1);
  const int C = (int)c.C, W = (int)c.W, H = (int)c.H;
  const bool two = ch + 1 < C;
  const int grows = g.band + D, xrows = g.band * S;
  const int grow = g.gc * GP, xrow = g.xc * XP;
  const uint32_t g_at = sm0 + (la * grows * g.gc + ls * (PX / S)) * GP + pl * (GP / CT);
  const uint32_t x_at = sm0 + g.x_at + (la * xrows * g.xc + ls * PX) * XP + pl * (XP / CT);
  if (threadIdx.x == 0) {
    for (int i = 0; i < g.stages; ++i) tma::mbar_init(&full[i], 1);
    tma::fence_init();
  }
  __syncthreads();

  struct Item {
    int n0, v0, tb;
  };
  auto item_of = [&](int i) {
    Item it;
    uint32_t q, n;
    const uint32_t seg = g.d_segs.divmod((uint32_t)i, q);
    const uint32_t band = g.d_bands.divmod(q, n);
    it.n0 = (int)n * g.ns;
    it.v0 = g.v_begin + (int)seg * g.cs * PX;
    it.tb = g.t_begin + (int)band * g.band;
    return it;
  };
  int p_item = chunk, p_slot = 0;
  auto issue = [&]() {
    if (p_item >= g.items) return;
    const Item it = item_of(p_item);
    unsigned char* const slot = smdyn + base + p_slot * g.stage_bytes;
    const bool bring_x = GW && g.want_x;
    tma::fence_async_smem();
    tma::mbar_expect_tx(&full[p_slot], (uint32_t)(g.gy_bytes + (bring_x ? g.x_bytes : 0)));
    tma::load_4d(slot, map_gy, ch0, it.v0 / S - D, it.tb - D, it.n0, &full[p_slot]);
    if (bring_x) tma::load_4d(slot + g.x_at, map_x, kCode ? ch0 / 2 : ch0, it.v0 - c.pw, it.tb * S - c.ph, it.n0, &full[p_slot]);
    p_slot = p_slot + 1 == g.stages ? 0 : p_slot + 1;
    p_item += g.chunks;
  };
  wait_for_previous();  // the aligned copies of the same call, where there are any
  if (threadIdx.x == 0)
    for (int i = 0; i < g.stages - 1; ++i) issue();

  f32x2 acc[K * K + (GW ? 1 : 0)];  // the filter, or its gradient and the bias's
#pragma unroll
  for (int k = 0; k < K * K + (GW ? 1 : 0); ++k) {
    acc[k] = 0;
    if (!GW && ch < C)
      acc[k] = pack_f32x2(ld(w + (int64_t)ch * K * K + k), two ? ld(w + (int64_t)(ch + 1) * K * K + k) : 0.f);
  }

  int slot = 0;
  uint32_t parity = 0;
  for (int item = chunk; item < g.items; item += g.chunks) {
    if (item > chunk) {  // the stage before this one is free once every thread is here
      __syncthreads();
      slot = slot + 1 == g.stages ? 0 : slot + 1;
      parity ^= slot == 0 ? 1u : 0u;
    }
    if (threadIdx.x == 0) issue();
    const Item it = item_of(item);
    const int64_t n = it.n0 + ln;
    const int strip = (it.v0 - g.v_begin) / PX + ls;
    const bool here = ln < g.ns && n < c.N && strip < g.strips, on = here && ch < C;
    const int iw0 = it.v0 + ls * PX - c.pw, ih0 = S * it.tb - c.ph;
    uint32_t xok = 0;
#pragma unroll
    for (int p = 0; p < PX; ++p) xok |= (iw0 + p >= 0 && iw0 + p < W) ? 1u << p : 0u;
    const int64_t at = n * H * (int64_t)W + (int64_t)ih0 * W + iw0;
    // a checkpoint's scales: lanes p + PX b of the strip's lanes read pixel p, block b of the tile's
    const int sb = (ch0 >> x8.shift) + pl / PX;
    const bool scaler = kCode && here && g.want_x && pl < 2 * PX && sb < x8.nblk && ((xok >> (pl % PX)) & 1);
    const int from = (int)(threadIdx.x & 31 & ~(CT - 1)) + PX * ((ch >> x8.shift) - (ch0 >> x8.shift));
    const float* const sp = x8.scales + (at + pl % PX) * x8.nblk + sb;
    if (!tma::mbar_wait(&full[slot], parity, timeouts)) {
      // the copy never landed: let those in flight finish (bounded), then stop
      for (int j = 1; j < g.stages; ++j) {
        const int q = (slot + j) % g.stages;
        tma::mbar_wait(&full[q], q > slot ? parity : parity ^ 1u, nullptr);
      }
      return;
    }
    uint32_t gs = g_at + slot * g.stage_bytes, xs = x_at + slot * g.stage_bytes;
    for (int t = 0; t < g.band; t += M, gs += M * grow, xs += RY * xrow) {
      f32x2 own[RY * PX];  // x of the strip, or its gx
#pragma unroll
      for (int r = 0; r < RY; ++r) {
        float sc = 0.f;
        if (kCode) {
          const int ih = ih0 + S * t + r;
          if (scaler && ih >= 0 && ih < H) sc = __ldg(sp + (int64_t)(S * t + r) * W * x8.nblk);
        }
#pragma unroll
        for (int p = 0; p < PX; ++p) {
          if constexpr (kCode) {
            Raw<T, SRC> v;
            v.s = __shfl_sync(0xffffffffu, sc, from + p);
            v.v = lds_u16(xs + r * xrow + p * XP);
            own[r * PX + p] = widen<T, SRC>(v);
          } else if constexpr (GW) {
            own[r * PX + p] = widen<T, SRC>(lds_pair<T>(xs + r * xrow + p * XP));
          } else {
            own[r * PX + p] = 0;
          }
        }
      }
      if (!on) continue;
      uint32_t q = gs;
#pragma unroll
      for (int e = -D; e <= (RY - 1) / S; ++e, q += grow) {  // gy row t + e meets the filter's rows a = r - S e
        f32x2 gv[WIN];
#pragma unroll
        for (int j = 0; j < WIN; ++j) gv[j] = widen<T, kSrcFull>(lds_pair<T>(q + j * GP));
#pragma unroll
        for (int r = 0; r < RY; ++r) {
          const int a = r - S * e;
          if (a < 0 || a >= K) continue;
#pragma unroll
          for (int m = 0; m < K * PX; ++m) {  // neighbouring products go to different sums
            const int b = GW ? m % K : m / PX, p = GW ? m / K : m % PX;
            if ((p - b) % S != 0) continue;
            const f32x2 v = gv[D + (p - b) / S];
            if (GW) {
              fma_f32x2(acc[a * K + b], own[r * PX + p], v);
              if (a == K / 2 && b == K / 2) acc[K * K] = add_f32x2(acc[K * K], v);
            } else {
              fma_f32x2(own[r * PX + p], acc[a * K + b], v);
            }
          }
        }
      }
      if (!GW) {
#pragma unroll
        for (int r = 0; r < RY; ++r) {
          const int ih = ih0 + S * t + r;
          if (ih < 0 || ih >= H) continue;
          T* o = gx + (at + (int64_t)(S * t + r) * W) * C + ch;
          if (g.pair_out) store_strip<T, true, PX>(o, C, own + r * PX, xok, true, g.accumulate);
          else store_strip<T, false, PX>(o, C, own + r * PX, xok, two, g.accumulate);
        }
      }
    }
  }
  if constexpr (GW) join_lanes<NT, K * K + 1>(g.ct_log, acc, C, ch0, chunk, ws);
}

template <typename T, int SRC, int K, int S, int CT>
__global__ void __launch_bounds__(kTileThreads, K == 7 ? 3 : 4)
tile_kernel(Conv c, Staged g, const __grid_constant__ CUtensorMap map_gy, const __grid_constant__ CUtensorMap map_x,
            Act8 x8, unsigned int* timeouts, const T* __restrict__ w, T* __restrict__ gx, float* __restrict__ ws) {
  if (g.want_gw && blockIdx.y == 0)
    tile_walk<T, SRC, K, S, CT, true>(c, g, &map_gy, &map_x, x8, timeouts, w, gx, ws);
  else
    tile_walk<T, SRC, K, S, CT, false>(c, g, &map_gy, &map_x, x8, timeouts, w, gx, ws);
}

// ---- launches --------------------------------------------------------------

template <typename T, int SRC, bool PAIR>
cudaError_t launch(const Conv& c, const Geom& g, const T* x, const Act8& x8, const T* gy, const T* w, T* gx, float* ws,
                   cudaStream_t s) {
  const unsigned grid = (unsigned)(g.tiles * g.chunks);
  if (c.kh == 3) {
    if (c.sh == 1)
      ring3_kernel<T, SRC, 1, PAIR><<<grid, kRingThreads, 0, s>>>(c, g, x, x8, gy, w, gx, ws);
    else
      ring3_kernel<T, SRC, 2, PAIR><<<grid, kRingThreads, 0, s>>>(c, g, x, x8, gy, w, gx, ws);
    return cudaGetLastError();
  }
#define X(K, S)                                                                                       \
  if (c.kh == K && c.sh == S)                                                                         \
    block_kernel<T, SRC, K, S, PAIR>                                                                  \
        <<<dim3(grid, g.want_gx && g.want_gw ? 2 : 1), kBlockThreads, 0, s>>>(c, g, x, x8, gy, w, gx, ws);
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

template <typename T, int SRC, int K, int S, int CT>
cudaError_t launch_staged(const Conv& c, const Staged& g, const Views& v, const Act8& x8, const T* w, T* gx, float* ws,
                          cudaStream_t s) {
  CUtensorMap mg, mx;
  const uint64_t gd[4] = {(uint64_t)c.C, (uint64_t)c.Wo, (uint64_t)c.Ho, (uint64_t)c.N};
  const uint64_t gs[3] = {(uint64_t)v.gdist, (uint64_t)(c.Wo * v.gdist), (uint64_t)(c.Ho * c.Wo * v.gdist)};
  const uint32_t gb[4] = {2 * CT, (uint32_t)g.gc, (uint32_t)g.grows, (uint32_t)g.ns};
  // codes go as 16-bit pairs (an odd last channel's partner is read and not used)
  constexpr uint64_t kPer = SRC == kSrcFull ? 1 : 2;
  const uint64_t xd[4] = {((uint64_t)c.C + kPer - 1) / kPer, (uint64_t)c.W, (uint64_t)c.H, (uint64_t)c.N};
  const uint64_t xs[3] = {(uint64_t)v.xdist, (uint64_t)(c.W * v.xdist), (uint64_t)(c.H * c.W * v.xdist)};
  const uint32_t xb[4] = {(uint32_t)(2 * CT / kPer), (uint32_t)g.xc, (uint32_t)g.xrows, (uint32_t)g.ns};
  if (!tma::encode_strided(&mg, v.gy, c.dtype, 4, gd, gs, gb)) return cudaErrorNotSupported;
  mx = mg;
  if (g.want_x && !tma::encode_strided(&mx, v.x, SRC == kSrcFull ? c.dtype : (int)DWCONV_F16, 4, xd, xs, xb))
    return cudaErrorNotSupported;
  unsigned int* to = tma::timeout_counter();
  if (!to) return cudaErrorNotSupported;
  const int smem = g.stages * g.stage_bytes + 128;
  auto go = [&](auto kern, unsigned sides) {
    // one limit for every shape: calls from several threads do not lower each other's
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(g.tiles * g.chunks), sides);
    if (v.copied) return launch_dependent(kern, grid, dim3(g.threads), (size_t)smem, s, c, g, mg, mx, x8, to, w, gx, ws);
    kern<<<grid, g.threads, smem, s>>>(c, g, mg, mx, x8, to, w, gx, ws);
    return cudaGetLastError();
  };
  if constexpr (K == 3) {
    return go(staged3_kernel<T, SRC, S, CT>, 1);
  } else {
    return go(tile_kernel<T, SRC, K, S, CT>, g.want_gx && g.want_gw ? 2 : 1);
  }
}

template <typename T>
cudaError_t run_staged(const Conv& c, const Staged& g, int src, const Views& v, const Act8& x8, const T* w, T* gx,
                       float* ws, cudaStream_t s) {
  // copies start on 16 bytes: pointers, distances between pixels
  auto fits = [](const void* p, int64_t dist) { return p && reinterpret_cast<uintptr_t>(p) % 16 == 0 && dist % 16 == 0; };
  if (!fits(v.gy, v.gdist) || (g.want_x && !fits(v.x, v.xdist))) return cudaErrorNotSupported;
#define X(SRC, K, S, CT)                                             \
  if (src == SRC && c.kh == K && c.sh == S && (1 << g.ct_log) == CT) \
    return launch_staged<T, SRC, K, S, CT>(c, g, v, x8, w, gx, ws, s);
#define Z(SRC, K) X(SRC, K, 1, 32) X(SRC, K, 2, 32) X(SRC, K, 1, 16) X(SRC, K, 2, 16)
#define Y(SRC) Z(SRC, 3) Z(SRC, 5) Z(SRC, 7)
  Y(kSrcFull) Y(kSrcI8) Y(kSrcE4M3)
#undef Y
#undef Z
#undef X
  return cudaErrorNotSupported;
}

}  // namespace walk
}  // namespace nhwc
}  // namespace dwconv
