// Channels-last (NHWC) backward: gx, gw and gb from gy, w and the layer's
// input, in full or from its 8-bit checkpoint.
//
//   gx[n, i, j, c] = sum_{m, a, b} w[c*m, a, b] gy[n, (i + ph - a*dh) / sh, (j + pw - b*dw) / sw, c*m]
//   gw[oc, a, b]   = sum_{n, o, q} gy[n, o, q, oc] x[n, o*sh - ph + a*dh, q*sw - pw + b*dw, oc / m]
//   gb[oc]         = sum_{n, o, q} gy[n, o, q, oc]
//
// The row-walking kernels (nhwc_bwd_impl.cuh) serve square 3x3, 5x5 and 7x7
// filters; the generic kernels here serve every descriptor: gx with one value
// per thread, gw with one block per (channels, tap, chunk of output pixels)
// and partial sums that a second launch adds in chunk order.
#include "dependent.cuh"
#include "nhwc_bwd.h"
#include "vec.cuh"

namespace dwconv {
namespace nhwc {
namespace {

constexpr int kNT = 256;

template <typename T>
__global__ void __launch_bounds__(kNT)
gx_generic_kernel(Conv c, int64_t total, const T* __restrict__ gy, const T* __restrict__ w, T* gx, bool accumulate) {
  for (int64_t i = blockIdx.x * (int64_t)kNT + threadIdx.x; i < total; i += (int64_t)gridDim.x * kNT) {
    const int64_t ch = i % c.C;
    int64_t r = i / c.C;
    const int64_t iw = r % c.W;
    r /= c.W;
    const int64_t ih = r % c.H;
    const int64_t n = r / c.H;
    float acc = 0.f;
    for (int a = 0; a < c.kh; ++a) {
      const int64_t th = ih + c.ph - (int64_t)a * c.dh;
      if (th < 0 || th % c.sh != 0 || th / c.sh >= c.Ho) continue;
      for (int b = 0; b < c.kw; ++b) {
        const int64_t tw = iw + c.pw - (int64_t)b * c.dw;
        if (tw < 0 || tw % c.sw != 0 || tw / c.sw >= c.Wo) continue;
        const T* g = gy + ((n * c.Ho + th / c.sh) * c.Wo + tw / c.sw) * c.ctot + c.off + ch * c.m;
        const T* wp = w + (ch * c.m * c.kh + a) * c.kw + b;
        for (int j = 0; j < c.m; ++j) acc = fmaf(ld(wp + (int64_t)j * c.kh * c.kw), ld(g + j), acc);
      }
    }
    if (accumulate) acc += ld_rw(gx + i);
    gx[i] = from_f<T>(acc);
  }
}

template <typename T, int SRC>
__device__ __forceinline__ float input_at(const T* x, const Act8& t, int64_t row, int64_t C, int64_t ch) {
  if constexpr (SRC == kSrcFull) {
    return ld(x + row * C + ch);
  } else {
    return __fmul_rn(code1<SRC>(t.codes[row * C + ch]), __ldg(t.scales + row * t.nblk + (ch >> t.shift)));
  }
}

// ws[chunk][oc][tap] (tap == taps: bias): 32 channels x 8 pixel lanes per block
template <typename T, int SRC>
__global__ void __launch_bounds__(kNT)
gw_generic_kernel(Conv c, int64_t pixels, int64_t per_chunk, const T* __restrict__ x, Act8 t,
                  const T* __restrict__ gy, float* __restrict__ ws, bool want_w, bool want_b) {
  __shared__ float sm[kNT];
  const int taps = c.kh * c.kw;
  const int tap = blockIdx.y;
  if (tap < taps ? !want_w : !want_b) return;
  const int64_t oc = blockIdx.x * (int64_t)32 + (threadIdx.x & 31);
  const int64_t OC = c.C * c.m;
  const int64_t p0 = blockIdx.z * per_chunk;
  const int64_t p1 = min(p0 + per_chunk, pixels);
  float acc = 0.f;
  if (oc < OC) {
    const int64_t a = (int64_t)(tap / c.kw) * c.dh - c.ph, b = (int64_t)(tap % c.kw) * c.dw - c.pw;
    for (int64_t p = p0 + (threadIdx.x >> 5); p < p1; p += kNT / 32) {
      const float g = ld(gy + p * c.ctot + c.off + oc);
      if (tap == taps) {
        acc += g;
        continue;
      }
      const int64_t q = p % c.Wo, o = p / c.Wo;
      const int64_t n = o / c.Ho;
      const int64_t ih = (o - n * c.Ho) * c.sh + a, iw = q * c.sw + b;
      if (ih < 0 || ih >= c.H || iw < 0 || iw >= c.W) continue;
      acc = fmaf(g, input_at<T, SRC>(x, t, (n * c.H + ih) * c.W + iw, c.C, oc / c.m), acc);
    }
  }
  sm[threadIdx.x] = acc;
  __syncthreads();
  if (threadIdx.x < 32 && oc < OC) {
    for (int i = 1; i < kNT / 32; ++i) acc += sm[i * 32 + threadIdx.x];
    ws[(blockIdx.z * OC + oc) * (taps + 1) + tap] = acc;
  }
}

int64_t out_pixels(const Conv& c) { return c.N * c.Ho * c.Wo; }

// Chunks of output pixels: enough blocks to fill the GPU, at least 64 pixels
// each, partial sums of at most 64 MB where that leaves two chunks or more;
// and no more than 1024 pixels of a lane, as far as 4096 chunks and 1 GB go,
// since a chain of n additions of like terms can be off by n / 4 * 2^-24 of
// the sum. (64x56x56x128 9x9 bf16 from codes: 19.3 ms with the last rule, 20.6
// without; a second sum inside the kernel cost 4 to 12 % of the call.)
int generic_chunks(const Conv& c) {
  if (c.N == 0) return 0;
  const int64_t taps1 = (int64_t)c.kh * c.kw + 1, one = c.C * c.m * taps1 * 4;
  const int64_t blocks = (c.C * c.m + 31) / 32 * taps1;
  int64_t n = (152 * 8 + blocks - 1) / blocks;
  const int64_t most = (out_pixels(c) + 63) / 64;
  const int64_t room = (int64_t(64) << 20) / one, wide = (int64_t(1) << 30) / one;
  if (n > most) n = most;
  if (n > room) n = room;
  constexpr int64_t kRun = 1024 * (kNT / 32);
  int64_t runs = (out_pixels(c) + kRun - 1) / kRun;
  if (runs > wide) runs = wide;
  if (runs > 4096) runs = 4096;  // a second pass adds them up in one chain
  if (n < runs) n = runs;
  if (n < 1) n = 1;
  return (int)n;
}

template <typename T>
cudaError_t generic(const Conv& c, const T* x, const Act8& t, const T* gy, const T* w, T* gx, T* gw, T* gb,
                    bool accumulate, float* ws, cudaStream_t s) {
  const int64_t OC = c.C * c.m;
  if (gx && c.N > 0) {
    const int64_t total = c.N * c.H * c.W * c.C;
    const int64_t blocks = (total + kNT - 1) / kNT;
    gx_generic_kernel<T><<<(unsigned)(blocks < 152 * 64 ? blocks : 152 * 64), kNT, 0, s>>>(c, total, gy, w, gx,
                                                                                           accumulate);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (!gw && !gb) return cudaSuccess;
  const int chunks = generic_chunks(c);
  if (chunks > 0) {
    const int64_t pixels = out_pixels(c);
    const int64_t per = (pixels + chunks - 1) / chunks;
    const dim3 grid((unsigned)((OC + 31) / 32), (unsigned)(c.kh * c.kw + 1), (unsigned)chunks);
    if (x || !t.codes)
      gw_generic_kernel<T, kSrcFull><<<grid, kNT, 0, s>>>(c, pixels, per, x, t, gy, ws, gw != nullptr, gb != nullptr);
    else if (t.src == kSrcI8)
      gw_generic_kernel<T, kSrcI8><<<grid, kNT, 0, s>>>(c, pixels, per, x, t, gy, ws, gw != nullptr, gb != nullptr);
    else
      gw_generic_kernel<T, kSrcE4M3><<<grid, kNT, 0, s>>>(c, pixels, per, x, t, gy, ws, gw != nullptr, gb != nullptr);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return bwd_weight_pass2(c, ws, chunks, gw, gb, s);
}

// gw and gb from the row-walking kernels' sums ws[chunk][tap][channel]: 32
// channels of one tap per block, a warp for every 32nd chunk
constexpr int kJoin = 1024;
template <typename T>
__global__ void __launch_bounds__(kJoin)
walk_join_kernel(int C, int taps, int chunks, const float* __restrict__ ws, T* __restrict__ gw, T* __restrict__ gb) {
  __shared__ float sm[kJoin];
  wait_for_previous();
  const int tap = blockIdx.y;
  if (tap < taps ? gw == nullptr : gb == nullptr) return;
  const int ch = blockIdx.x * 32 + (threadIdx.x & 31);
  float acc = 0.f;
  if (ch < C) {
#pragma unroll 8
    for (int k = threadIdx.x >> 5; k < chunks; k += kJoin / 32) acc += ws[((int64_t)k * (taps + 1) + tap) * C + ch];
  }
  sm[threadIdx.x] = acc;
  __syncthreads();
  if (threadIdx.x < 32 && ch < C) {
#pragma unroll
    for (int i = 1; i < kJoin / 32; ++i) acc += sm[i * 32 + threadIdx.x];
    if (tap < taps) gw[(int64_t)ch * taps + tap] = from_f<T>(acc);
    else gb[ch] = from_f<T>(acc);
  }
}

template <typename T>
cudaError_t direct(const Conv& c, const T* x, const Act8& t, const T* gy, const T* w, T* gx, bool want_gw,
                   bool accumulate, float* ws, cudaStream_t s, int* chunks) {
  walk::Geom g = walk::plan(c);
  g.want_gx = gx != nullptr;
  g.want_gw = want_gw;
  g.accumulate = accumulate;
  *chunks = g.chunks;
  auto even = [](const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; };
  const bool pair = c.C % 2 == 0 && c.ctot % 2 == 0 && c.off % 2 == 0 && even(x, 2 * sizeof(T)) &&
                    even(gy, 2 * sizeof(T)) && even(gx, 2 * sizeof(T)) && even(t.codes, 2);
  return walk::run<T>(c, g, pair, x, t, gy, w, gx, ws, s);
}

// Pixels of `bytes` bytes, `from` apart, copied `to` apart (a multiple of 16):
// the layout that the staged kernels read. A thread writes 16 bytes; their
// source begins anywhere, so it is read as aligned words and shifted. The
// detour pays: 10x17x52x287 fp16 5x5 takes 27 us with it, 111 without (every
// access of two channels being two).
struct Copy {
  const uint8_t* src;
  uint8_t* dst;
  int64_t pixels, from, to;
  int bytes;
  FastDiv d_vecs;   // 16-byte vectors of a pixel
};

// The five aligned words that hold the 16 bytes at `src`, from reads inside [lo, end) alone: next to either end the words
// are put together from their bytes there, the others being 0.
struct GlobalBytes {
  static __device__ __forceinline__ uint32_t word(const uint8_t* p) { return __ldg(reinterpret_cast<const uint32_t*>(p)); }
  static __device__ __forceinline__ uint32_t byte(const uint8_t* p) { return __ldg(p); }
};
#pragma nv_exec_check_disable
template <typename Load>
__host__ __device__ __forceinline__ void words_at(const uint8_t* src, const uint8_t* lo, const uint8_t* end, uint32_t* v) {
  const uint8_t* q = src - (reinterpret_cast<uintptr_t>(src) & 3);
  if (q >= lo && end - q >= 20) {
#pragma unroll
    for (int e = 0; e < 5; ++e) v[e] = Load::word(q + 4 * e);
  } else {
#pragma unroll
    for (int e = 0; e < 5; ++e) {
      uint32_t w = 0;
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {
        const uint8_t* const p = q + 4 * e + b;
        if (p >= lo && p < end) w |= Load::byte(p) << (8 * b);
      }
      v[e] = w;
    }
  }
}

__global__ void __launch_bounds__(kNT) align_kernel(Copy a, Copy b) {
  dependents_may_start();
  const Copy& k = blockIdx.y == 0 ? a : b;
  const int64_t total = k.pixels * k.d_vecs.d;
  const uint8_t* const end = k.src + (k.pixels - 1) * k.from + k.bytes;
  for (int64_t i = blockIdx.x * (int64_t)kNT + threadIdx.x; i < total; i += (int64_t)gridDim.x * kNT) {
    const int64_t p = i / k.d_vecs.d;
    const int at = (int)(i - p * k.d_vecs.d) * 16;
    const uint8_t* const src = k.src + p * k.from + at;
    const int shift = (int)(reinterpret_cast<uintptr_t>(src) & 3);
    uint32_t v[5];
    words_at<GlobalBytes>(src, k.src, end, v);
    uint4 o;
    o.x = __funnelshift_r(v[0], v[1], 8 * shift);
    o.y = __funnelshift_r(v[1], v[2], 8 * shift);
    o.z = __funnelshift_r(v[2], v[3], 8 * shift);
    o.w = __funnelshift_r(v[3], v[4], 8 * shift);
    *reinterpret_cast<uint4*>(k.dst + p * k.to + at) = o;
  }
}

int64_t up16(int64_t v) { return (v + 15) / 16 * 16; }

// Bytes of aligned copies of gy and of x that a descriptor needs (0: as they are); x8: of its codes.
int64_t gy_copy_bytes(const Conv& c, int es) {
  return c.ctot * es % 16 == 0 && c.off * es % 16 == 0 ? 0 : out_pixels(c) * up16(c.C * es);
}
int64_t x_copy_bytes(const Conv& c, int es) {
  return c.C * es % 16 == 0 ? 0 : c.N * c.H * c.W * up16(c.C * es);
}
// Copies of more than this are not made: the direct kernels run.
constexpr int64_t kMostCopy = int64_t(4) << 30;

bool copies_fit(const Conv& c, int es) {
  return gy_copy_bytes(c, es) + x_copy_bytes(c, es) <= kMostCopy && gy_copy_bytes(c, es) + x_copy_bytes(c, 1) <= kMostCopy;
}

size_t sums_bytes(const Conv& c, int64_t chunks) {
  const size_t b = (size_t)chunks * (size_t)c.OC() * (size_t)(c.kh * c.kw + 1) * sizeof(float);
  return (b + 255) & ~size_t(255);
}
// The staged plan of a call from this source and the bytes of its aligned copies of gy and of x (or its codes): what the
// workspace is sized by and what a call lays out in it. A source's plan says nothing of another's: a stage of codes is
// smaller than one of full values, and on tall images only it may fit. false: the direct kernels run.
struct Copies {
  int64_t gy, x;
};
bool staged_of(const Conv& c, int src, walk::Staged* g, Copies* k) {
  const int es = c.dtype == DWCONV_F32 ? 4 : 2;
  if (!walk::plan_staged(c, src, g) || !copies_fit(c, es)) return false;
  *k = Copies{gy_copy_bytes(c, es), x_copy_bytes(c, src == kSrcFull ? es : 1)};
  return true;
}

// chunks of any of the walking kernels that a call's pointers and source may lead to
int64_t walk_chunks(const Conv& c) {
  int64_t n = walk::plan(c).chunks;
  for (int src : {kSrcFull, kSrcI8}) {
    walk::Staged g;
    if (walk::plan_staged(c, src, &g) && g.chunks > n) n = g.chunks;
  }
  return n;
}

template <typename T>
cudaError_t walked(const Conv& c, const T* x, const Act8& t, const T* gy, const T* w, T* gx, T* gw, T* gb,
                   bool accumulate, float* ws, cudaStream_t s) {
  const bool want_gw = gw != nullptr || gb != nullptr;
  const int taps = c.kh * c.kw;
  int chunks = 0;
  walk::Staged st;
  cudaError_t e = cudaErrorNotSupported;
  const int src = x || !t.codes ? kSrcFull : t.src, es = sizeof(T), xes = src == kSrcFull ? es : 1;
  Copies need;
  // gx alone has no workspace, so no copies
  if (staged_of(c, src, &st, &need) && (want_gw || need.gy == 0)) {
    const int64_t gcopy = need.gy, xcopy = gw ? need.x : 0;
    st.want_gx = gx != nullptr;
    st.want_gw = want_gw;
    st.want_x = gw != nullptr;
    st.accumulate = accumulate;
    st.pair_out = c.C % 2 == 0 && reinterpret_cast<uintptr_t>(gx) % (2 * es) == 0;
    chunks = st.chunks;
    walk::Views v{gy + c.off, src == kSrcFull ? (const void*)x : t.codes, c.ctot * es, c.C * xes, false};
    uint8_t* room = reinterpret_cast<uint8_t*>(ws) + (gcopy || xcopy ? sums_bytes(c, walk_chunks(c)) : 0);
    Copy job[2] = {};
    int jobs = 0;
    auto copy = [&](const void** p, int64_t* dist, int64_t pixels, int64_t bytes) {
      const int64_t to = up16(bytes);
      job[jobs++] = Copy{(const uint8_t*)*p, room, pixels, *dist, to, (int)bytes, FastDiv((uint32_t)(to / 16))};
      *p = room;
      *dist = to;
      room += pixels * to;
    };
    if (gcopy) copy(&v.gy, &v.gdist, out_pixels(c), c.C * es);
    if (xcopy) copy(&v.x, &v.xdist, c.N * c.H * c.W, c.C * xes);
    if (jobs) {
      const int64_t most = (gcopy > xcopy ? gcopy : xcopy) / 16;
      const int64_t blocks = (most + kNT - 1) / kNT;
      align_kernel<<<dim3((unsigned)(blocks < 152 * 32 ? blocks : 152 * 32), (unsigned)jobs), kNT, 0, s>>>(job[0], job[1]);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
      v.copied = true;
    }
    e = walk::run_staged<T>(c, st, src, v, t, w, gx, ws, s);
  }
  if (e == cudaErrorNotSupported) e = direct<T>(c, x, t, gy, w, gx, want_gw, accumulate, ws, s, &chunks);
  if (e != cudaSuccess || !want_gw) return e;
  return launch_dependent(walk_join_kernel<T>, dim3((unsigned)((c.C + 31) / 32), (unsigned)(taps + 1)), dim3(kJoin), 0, s,
                          (int)c.C, taps, chunks, (const float*)ws, gw, gb);
}

}  // namespace

namespace walk {

// Padding of at most (K - 1) / 2 makes every output's centre tap an input
// position (see nhwc_bwd_impl.cuh); sides and channels are indexed in 32 bits.
bool supported(const Conv& c) {
  if (c.kh != c.kw || (c.kh != 3 && c.kh != 5 && c.kh != 7)) return false;
  if (c.sh != c.sw || c.sh > 2 || c.dh != 1 || c.dw != 1 || c.m != 1) return false;
  if (c.ph > c.kh / 2 || c.pw > c.kw / 2) return false;
  return c.H < (1 << 28) && c.W < (1 << 28) && c.C <= (1 << 20) && c.N > 0;
}

Geom plan(const Conv& c) {
  Geom g{};
  const int K = c.kh, S = c.sh;
  const bool ring = K == 3;
  const int px = ring ? 4 : 8, nt = ring ? kRingThreads : kBlockThreads, step = ring ? 1 : 2 / S;
  // 64 channels per block, 32 where that leaves a quarter fewer of the last tile idle, fewer for few channels
  const int64_t by64 = (c.C + 63) / 64 * 64, by32 = (c.C + 31) / 32 * 32, pairs = (c.C + 1) / 2;
  g.ct_log = 4 * by64 >= 5 * by32 ? 4 : 5;
  while (g.ct_log > 0 && (int64_t(1) << (g.ct_log - 1)) >= pairs) --g.ct_log;
  const int ct = 1 << g.ct_log, lanes = nt >> g.ct_log;
  g.tiles = (int)((pairs + ct - 1) / ct);
  g.t_begin = c.ph / S;
  g.t_end = (int)((c.H + c.ph - 1) / S) + 1;
  g.v_begin = c.pw / S * S;
  g.strips = (int)((c.W + c.pw - g.v_begin + px - 1) / px);
  // Bands of rows: the cut whose longest block has the least to do, a band costing its steps and, where rows of gy stay
  // in registers, those read above it. gx and gw of the larger filters run side by side.
  const int64_t wave = ring ? 152 * kRingBlocks : 152 * kBlockBlocks / 2;
  const int64_t per_tile = (wave + g.tiles - 1) / g.tiles;
  const int64_t rows = g.t_end - g.t_begin;
  const double above = ring ? 0.75 * (2 / S) + 0.5 : 0.25;
  double best = -1;
  for (int64_t bands = 1; bands <= (rows + step - 1) / step && bands <= 512; ++bands) {
    int64_t band = (rows + bands - 1) / bands;
    band = (band + step - 1) / step * step;
    const int64_t items = c.N * ((rows + band - 1) / band) * g.strips, groups = (items + lanes - 1) / lanes;
    const double cost = (double)((groups + per_tile - 1) / per_tile) * ((double)band / step + above);
    if (best >= 0 && cost >= best) continue;
    best = cost;
    g.band = (int)band;
    g.bands = (int)((rows + band - 1) / band);
    g.items = items;
    g.groups = groups;
  }
  // one wave of blocks, more where a thread would add up over 4096 products per filter value
  int64_t chunks = per_tile;
  const int64_t long_chain = g.groups * g.band * px / 4096;
  if (chunks < long_chain) chunks = long_chain;
  if (chunks > g.groups) chunks = g.groups;
  const int64_t room = (int64_t(1) << 30) / (c.C * (K * K + 1) * 4);  // at most 1 GB of partial sums
  if (chunks > room) chunks = room < 1 ? 1 : room;
  g.chunks = (int)chunks;
  return g;
}

bool plan_staged(const Conv& c, int src, Staged* out) {
  if (!supported(c) || c.N >= (int64_t(1) << 31)) return false;
  const int es = c.dtype == DWCONV_F32 ? 4 : 2, K = c.kh, S = c.sh, D = (K - 1) / S;
  const bool ring = K == 3;
  const int px = ring ? 4 : tile_px(K), step = ring ? 1 : 2 / S, blocks = ring ? kStagedBlocks : K == 5 ? 4 : 3;
  // A tile has 32 channels at least. With fewer the direct kernels' narrower blocks win sooner or later: 3x3 bf16 at 64
  // samples, 8 channels 23 us (direct) against 56 (staged), 24 the same; 5x5 bf16, 24 channels 39 against 23, 9 channels 49
  // against 31; 7x7, 17 channels 117 against 64, 12 channels 29 against 31: one bound for both serves 7x7 with 9 to about
  // 12 channels a little worse.
  if (c.C < (K == 3 ? 24 : 9)) return false;
  // The 3x3 kernel steps from a row's scales to the next row's by 32 bits of bytes: longer rows (2^35 values from blocks
  // of 32) take the direct kernel.
  if (ring && src != kSrcFull && c.W * ((c.C + 31) / 32) * 4 >= (int64_t(1) << 32)) return false;
  Staged g{};
  // 64 channels per block, 32 where that leaves a quarter fewer of the last tile idle
  const int64_t by64 = (c.C + 63) / 64 * 64, by32 = (c.C + 31) / 32 * 32;
  g.ct_log = 4 * by64 >= 5 * by32 ? 4 : 5;
  const int ct = 1 << g.ct_log, most = (ring ? kStagedThreads : kTileThreads) / ct;
  g.tiles = (int)((c.C + 2 * ct - 1) / (2 * ct));
  g.t_begin = c.ph / S;
  g.t_end = (int)((c.H + c.ph - 1) / S) + 1;
  g.v_begin = c.pw / S * S;
  g.strips = (int)((c.W + c.pw - g.v_begin + px - 1) / px);
  const int xes = src == kSrcFull ? es : 1;
  // Strips and samples of a block's lanes: the split that leaves the fewest lanes idle, a narrow block paying for the
  // columns of gy that it shares with its neighbours.
  double fit = -1;
  for (int cs = 1; cs <= most && cs <= g.strips; ++cs) {
    const int segs = (g.strips + cs - 1) / cs;
    const int64_t ns = most / cs < c.N ? most / cs : c.N, groups = (c.N + ns - 1) / ns;
    const double busy = (double)g.strips * c.N * ct / ((double)segs * groups * ((cs * ns * ct + 31) / 32 * 32));
    const double f = busy * (cs * ns * ct >= 96 ? 1.0 : 0.7) / (1 + 0.15 * D * S / (cs * px));
    if (f <= fit) continue;
    fit = f;
    g.cs = cs;
    g.segs = segs;
    g.ns = (int)ns;
  }
  g.threads = (g.cs * g.ns * ct + 31) / 32 * 32;
  g.gc = D + (g.cs * px - 1) / S + 1;
  g.xc = g.cs * px;
  const int room = 220 * 1024 / blocks - 6 * 1024;  // of a block; 6 KB: what join_lanes keeps
  auto stage = [&](Staged* q, int grows, int xrows) {
    q->grows = grows;
    q->xrows = xrows;
    q->gy_bytes = q->ns * grows * q->gc * 2 * ct * es;
    q->x_bytes = q->ns * xrows * q->xc * 2 * ct * xes;
    q->x_at = (q->gy_bytes + 127) / 128 * 128;
    q->stage_bytes = (q->x_at + q->x_bytes + 127) / 128 * 128;
  };
  // Bands: the cut whose longest block has the fewest rows. A band of the 3x3 kernel costs whole stages, the rows above
  // it about a third of an owned row; one of the larger filters is a stage, whose copy and start cost about half a step.
  // Cuts into over 4096 bands are not looked at, so that planning stays within tens of microseconds: images whose rows
  // need more (a large filter's stage holds at most four steps) take the direct kernels.
  const int64_t rows = g.t_end - g.t_begin, groups = (c.N + g.ns - 1) / g.ns;
  const int rd = D + 1;
  const int64_t wave = (152 * blocks / (ring ? 1 : 2) + g.tiles - 1) / g.tiles;
  double best = -1;
  for (int64_t bands = 1; bands <= rows && bands <= 4096; ++bands) {
    int64_t band = (rows + bands - 1) / bands;
    if (!ring) band = (band + step - 1) / step * step;
    if ((rows + band - 1) / band != bands) continue;
    if (!ring) {
      if (band > 4 * step) continue;
      stage(&g, (int)band + D, (int)band * S);
      if (g.stage_bytes > room && band > step) continue;
      if (g.stage_bytes + 128 > kMostSmem) continue;
    }
    const int64_t items = groups * g.segs * bands;
    if (items >= (1 << 30)) break;
    const double one = ring ? (D + band + rd - 1) / rd * rd - 0.7 * D + 0.5 : (double)band / step + 0.5;
    const double cost = (double)((items + wave - 1) / wave) * one;
    if (best < 0 || cost < best) {
      best = cost;
      g.bands = (int)bands;
      g.band = (int)band;
      g.items = (int)items;
    }
  }
  if (best < 0) return false;
  if (ring) {
    stage(&g, rd, rd * S);
    g.stages = room / g.stage_bytes;
    if (g.stages < 2) g.stages = 2;
  } else {
    stage(&g, g.band + D, g.band * S);
    g.stages = room / g.stage_bytes;
    if (g.stages < 1) g.stages = 1;
    if (g.stages > 2) g.stages = 2;
  }
  if (g.stages > kMaxStages) g.stages = kMaxStages;
  if (g.stages * g.stage_bytes + 128 > kMostSmem) return false;
  g.d_segs = FastDiv((uint32_t)g.segs);
  g.d_bands = FastDiv((uint32_t)g.bands);
  int64_t chunks = g.items < wave ? g.items : wave;
  const int64_t long_chain = (int64_t)g.items * g.band * px * S / 4096;  // at most 4096 products in a thread's chain
  if (chunks < long_chain) chunks = long_chain < g.items ? long_chain : g.items;
  const int64_t most_chunks = (int64_t(1) << 30) / (c.C * (K * K + 1) * 4);
  if (chunks > most_chunks) chunks = most_chunks < 1 ? 1 : most_chunks;
  g.chunks = (int)chunks;
  *out = g;
  return true;
}

}  // namespace walk

Algo plan_bwd(const Conv& c) { return walk::supported(c) ? Algo::Nhwc : Algo::Generic; }

size_t bwd_workspace_bytes(const Conv& c) {
  if (!walk::supported(c)) return sums_bytes(c, generic_chunks(c));
  size_t b = sums_bytes(c, walk_chunks(c));
  int64_t most = 0;
  for (int src : {kSrcFull, kSrcI8}) {
    walk::Staged g;
    Copies k;
    if (staged_of(c, src, &g, &k) && k.gy + k.x > most) most = k.gy + k.x;
  }
  b += (size_t)most;
  return b;
}

cudaError_t bwd(const Conv& c, const void* x, const Act8& x8, const void* gy, const void* w, void* gx, void* gw,
                void* gb, bool accumulate, float* ws, cudaStream_t s) {
  cudaError_t e = cudaErrorInvalidValue;
  const bool walk = plan_bwd(c) == Algo::Nhwc;
  DWCONV_DISPATCH_DTYPE(c.dtype, T, e = walk ? walked<T>(c, (const T*)x, x8, (const T*)gy, (const T*)w, (T*)gx, (T*)gw,
                                                         (T*)gb, accumulate, ws, s)
                                             : generic<T>(c, (const T*)x, x8, (const T*)gy, (const T*)w, (T*)gx,
                                                          (T*)gw, (T*)gb, accumulate, ws, s));
  return e;
}

}  // namespace nhwc
}  // namespace dwconv
