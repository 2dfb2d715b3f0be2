// 8-bit activation checkpoints: encode and decode.
//
// Both are one pass over the data. A block of channels belongs to a group of
// neighbouring lanes of one warp, 16 bytes of x per lane: its maximum is a few
// shuffles, and x is read once. Rows that cannot be read 16 bytes at a time
// (channels, row distance or pointers not multiples of 16 bytes) take the
// element kernels, one warp per block.
//
// Bound by memory: 64x112x112x64 bf16 to e4m3 codes and back takes 52.5 us,
// 6.1 TB/s of the floor's 321 MB, 0.92 of the measured copy.
#include "act8.cuh"
#include "vec.cuh"

namespace dwconv {
namespace {

constexpr int kNT = 256;
// 16-byte vectors of a thread, all of them read before the first is used: four
// where there are many, one where two waves of blocks cover them all (45 x 51 x
// 200 fp32, three samples: 9.1 us for the round trip against 12.3 with four;
// 112 x 112 x 64 bf16, 64 samples: 52.5 us with four, 55.4 with two, 56.3 with
// eight).
constexpr int kMany = 4;
constexpr uint32_t kFew = 152 * 16 * kNT;

// Lanes: L = block / VEC per block; `per_row` = nblk * L vectors per row, the
// last ones of a ragged row idle.
struct EGeom {
  uint32_t total;  // vectors in this launch, below 2^31
  FastDiv d_row;   // vectors per row, idle ones included
  int64_t row0;    // first row of this launch
  int64_t ldx;
  int C, L;
};

template <typename T, int SRC, int kItems>
__global__ void __launch_bounds__(kNT) encode_kernel(EGeom g, const T* __restrict__ x, Act8 t) {
  constexpr int VEC = Vec<T>::n;
  const uint32_t base = blockIdx.x * (uint32_t)(kNT * kItems) + threadIdx.x;
  uint4 v[kItems];
  int64_t row[kItems];
  int c[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const uint32_t i = base + k * kNT;
    uint32_t q;
    const uint32_t r = g.d_row.divmod(i, q);
    row[k] = g.row0 + q;
    c[k] = i < g.total ? (int)r * VEC : g.C;  // g.C: idle
    v[k] = make_uint4(0, 0, 0, 0);
    if (c[k] < g.C) v[k] = __ldcs(reinterpret_cast<const uint4*>(x + row[k] * g.ldx + c[k]));
  }
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const uint32_t m = block_max<T, VEC>(v[k], g.L);  // a power of two of aligned lanes; idle lanes bring zeros
    if (c[k] >= g.C) continue;
    f32x2 f[VEC / 2];
    unpack16_pairs<T>(v[k], f);
    float inv;
    const float s = scale_of<SRC>(m, &inv);
    uint8_t* q = t.codes + row[k] * g.C + c[k];
    if constexpr (VEC == 8) {
      *reinterpret_cast<uint2*>(q) = make_uint2(encode4<SRC>(f[0], f[1], inv), encode4<SRC>(f[2], f[3], inv));
    } else {
      *reinterpret_cast<uint32_t*>(q) = encode4<SRC>(f[0], f[1], inv);
    }
    if ((c[k] & ((1 << t.shift) - 1)) == 0) t.scales[row[k] * t.nblk + (c[k] >> t.shift)] = s;
  }
}

// The blocks of channels of a warp: kWarpBlocks at a time, `step` of them
// further each time, as (row, block of the row) without a division per block.
constexpr int kWarpBlocks = 4;
struct BlockWalk {
  int64_t b, row;
  int blk;
  __device__ __forceinline__ void to(int64_t block, int nblk) {
    b = block;
    row = block / nblk;
    blk = (int)(block - row * nblk);
  }
  __device__ __forceinline__ void next(int nblk) {
    ++b;
    if (++blk == nblk) {
      blk = 0;
      ++row;
    }
  }
};

// A block of channels per warp, neighbouring lanes on neighbouring channels.
template <typename T, int SRC>
__global__ void __launch_bounds__(kNT)
encode_elem_kernel(int64_t rows, int C, int64_t ldx, const T* __restrict__ x, Act8 t) {
  const int lane = threadIdx.x & 31;
  const int64_t blocks = rows * t.nblk;
  const int64_t step = (int64_t)gridDim.x * (kNT / 32) * kWarpBlocks;
  BlockWalk w;
  for (int64_t b = (blockIdx.x * (int64_t)(kNT / 32) + (threadIdx.x >> 5)) * kWarpBlocks; b < blocks; b += step) {
    float f[kWarpBlocks][4];
    w.to(b, t.nblk);
#pragma unroll
    for (int u = 0; u < kWarpBlocks; ++u, w.next(t.nblk)) {
      const int c0 = w.blk << t.shift, n = w.b < blocks ? min(C - c0, 1 << t.shift) : 0;
      const T* p = x + w.row * ldx + c0;
#pragma unroll
      for (int j = 0; j < 4; ++j) f[u][j] = lane + 32 * j < n ? ld(p + lane + 32 * j) : 0.f;
    }
    w.to(b, t.nblk);
#pragma unroll
    for (int u = 0; u < kWarpBlocks; ++u, w.next(t.nblk)) {
      if (w.b >= blocks) break;
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) m = max(m, abs_bits(f[u][j]));
      m = __reduce_max_sync(0xffffffffu, m);
      float inv;
      const float s = scale_of<SRC>(m, &inv);
      const int c0 = w.blk << t.shift, n = min(C - c0, 1 << t.shift);
      uint8_t* q = t.codes + w.row * C + c0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (lane + 32 * j < n) q[lane + 32 * j] = encode1<SRC>(f[u][j], inv);
      if (lane == 0) t.scales[w.b] = s;
    }
  }
}

template <typename T, int SRC, int kItems>
__global__ void __launch_bounds__(kNT) decode_kernel(EGeom g, Act8 t, T* __restrict__ x) {
  constexpr int VEC = Vec<T>::n;
  const uint32_t base = blockIdx.x * (uint32_t)(kNT * kItems) + threadIdx.x;
  uint32_t v[kItems][2];
  float s[kItems];
  int64_t at[kItems];
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    const uint32_t i = base + k * kNT;
    at[k] = -1;
    if (i >= g.total) continue;
    uint32_t q;
    const uint32_t r = g.d_row.divmod(i, q);
    const int64_t row = g.row0 + q;
    const int c = (int)r * VEC;
    at[k] = row * g.ldx + c;
    const uint8_t* p = t.codes + row * g.C + c;
    if (VEC == 8) {
      const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p));
      v[k][0] = u.x;
      v[k][1] = u.y;
    } else {
      v[k][0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
    }
    s[k] = __ldg(t.scales + row * t.nblk + (c >> t.shift));
  }
#pragma unroll
  for (int k = 0; k < kItems; ++k) {
    if (at[k] < 0) continue;
    float f[VEC];
#pragma unroll
    for (int h = 0; h < VEC / 4; ++h) codes4<SRC>(v[k][h], f + 4 * h);
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = __fmul_rn(f[e], s[k]);
    *reinterpret_cast<uint4*>(x + at[k]) = pack16<T>(f);
  }
}

template <typename T, int SRC>
__global__ void __launch_bounds__(kNT)
decode_elem_kernel(int64_t rows, int C, int64_t ldx, Act8 t, T* __restrict__ x) {
  const int lane = threadIdx.x & 31;
  const int64_t blocks = rows * t.nblk;
  const int64_t step = (int64_t)gridDim.x * (kNT / 32) * kWarpBlocks;
  BlockWalk w;
  for (int64_t b = (blockIdx.x * (int64_t)(kNT / 32) + (threadIdx.x >> 5)) * kWarpBlocks; b < blocks; b += step) {
    uint8_t v[kWarpBlocks][4];
    float s[kWarpBlocks];
    w.to(b, t.nblk);
#pragma unroll
    for (int u = 0; u < kWarpBlocks; ++u, w.next(t.nblk)) {
      const int c0 = w.blk << t.shift, n = w.b < blocks ? min(C - c0, 1 << t.shift) : 0;
      const uint8_t* p = t.codes + w.row * C + c0;
      s[u] = n > 0 ? __ldg(t.scales + w.b) : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[u][j] = lane + 32 * j < n ? __ldg(p + lane + 32 * j) : 0;
    }
    w.to(b, t.nblk);
#pragma unroll
    for (int u = 0; u < kWarpBlocks; ++u, w.next(t.nblk)) {
      const int c0 = w.blk << t.shift, n = w.b < blocks ? min(C - c0, 1 << t.shift) : 0;
      T* p = x + w.row * ldx + c0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (lane + 32 * j < n) p[lane + 32 * j] = from_f<T>(__fmul_rn(code1<SRC>(v[u][j]), s[u]));
    }
  }
}

bool vec_ok(int64_t C, int64_t ldx, int es, const void* x, const Act8& t) {
  const int vec = 16 / es;
  return C % vec == 0 && ldx % vec == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
         reinterpret_cast<uintptr_t>(t.codes) % vec == 0;
}

unsigned grid_of(uint32_t vectors, int items) { return (vectors + kNT * items - 1) / (kNT * items); }

unsigned elem_grid(int64_t blocks) {
  const int64_t n = (blocks + kNT / 32 * kWarpBlocks - 1) / (kNT / 32 * kWarpBlocks);
  return (unsigned)(n < 152 * 32 ? n : 152 * 32);
}

// fn(geom) for launches of below 2^31 vectors each
template <typename F>
cudaError_t over_rows(int64_t rows, int64_t per_row, int64_t C, int64_t ldx, int L, F fn) {
  const int64_t most = ((int64_t(1) << 31) - kNT * kMany) / per_row;
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t n = rows - r < most ? rows - r : most;
    EGeom g{};
    g.total = (uint32_t)(n * per_row);
    g.d_row = FastDiv((uint32_t)per_row);
    g.row0 = r;
    g.ldx = ldx;
    g.C = (int)C;
    g.L = L;
    fn(g);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T, int SRC>
cudaError_t encode(int64_t rows, int64_t C, int64_t ldx, const T* x, const Act8& t, cudaStream_t s) {
  if (!vec_ok(C, ldx, sizeof(T), x, t)) {
    encode_elem_kernel<T, SRC><<<elem_grid(rows * t.nblk), kNT, 0, s>>>(rows, (int)C, ldx, x, t);
    return cudaGetLastError();
  }
  const int L = (1 << t.shift) / Vec<T>::n;
  return over_rows(rows, (int64_t)t.nblk * L, C, ldx, L, [&](const EGeom& g) {
    if (g.total > kFew) encode_kernel<T, SRC, kMany><<<grid_of(g.total, kMany), kNT, 0, s>>>(g, x, t);
    else encode_kernel<T, SRC, 1><<<grid_of(g.total, 1), kNT, 0, s>>>(g, x, t);
  });
}

template <typename T, int SRC>
cudaError_t decode(int64_t rows, int64_t C, int64_t ldx, const Act8& t, T* x, cudaStream_t s) {
  if (!vec_ok(C, ldx, sizeof(T), x, t)) {
    decode_elem_kernel<T, SRC><<<elem_grid(rows * t.nblk), kNT, 0, s>>>(rows, (int)C, ldx, t, x);
    return cudaGetLastError();
  }
  return over_rows(rows, C / Vec<T>::n, C, ldx, 0, [&](const EGeom& g) {
    if (g.total > kFew) decode_kernel<T, SRC, kMany><<<grid_of(g.total, kMany), kNT, 0, s>>>(g, t, x);
    else decode_kernel<T, SRC, 1><<<grid_of(g.total, 1), kNT, 0, s>>>(g, t, x);
  });
}

}  // namespace

cudaError_t act8_encode(int64_t rows, int64_t C, int64_t ldx, int dtype, const void* x, const Act8& t,
                        cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  cudaError_t e = cudaErrorInvalidValue;
  DWCONV_DISPATCH_DTYPE(dtype, T, e = t.src == kSrcI8 ? encode<T, kSrcI8>(rows, C, ldx, (const T*)x, t, s)
                                                      : encode<T, kSrcE4M3>(rows, C, ldx, (const T*)x, t, s));
  return e;
}

cudaError_t act8_decode(int64_t rows, int64_t C, int64_t ldx, int dtype, const Act8& t, void* x,
                        cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  cudaError_t e = cudaErrorInvalidValue;
  DWCONV_DISPATCH_DTYPE(dtype, T, e = t.src == kSrcI8 ? decode<T, kSrcI8>(rows, C, ldx, t, (T*)x, s)
                                                      : decode<T, kSrcE4M3>(rows, C, ldx, t, (T*)x, s));
  return e;
}

}  // namespace dwconv
