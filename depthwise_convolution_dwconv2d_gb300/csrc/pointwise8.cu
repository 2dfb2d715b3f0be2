// 1x1 layers over 8-bit floats: the weights' encoder, the choice of kernel,
// the aligned copy of codes, and a kernel for codes at any byte.
//
//   y[p, o] = act(sum_b sx[p, b] sw[o / 128, b] sum_{c in b} x[p, c] w[o, c] + bias[o])
//
// over blocks b of 128 channels. The sum within a block is one of products of
// e4m3 values, exact in fp32 but for the additions; each block's sum is
// multiplied by the product of its two scales and added in fp32.
#include "dependent.cuh"
#include "norm.cuh"
#include "pointwise8.h"
#include "vec.cuh"

namespace dwconv {
namespace pw8 {
namespace {

// ---- weights ----------------------------------------------------------------

// A block per 128 x 128 weights. It takes the maximum in a first read, encodes
// in a second (from L1 / L2), and writes whole rows of 128 codes, zeros behind
// the last channel, through shared memory. Weights are encoded once per
// change, so this is kept simple.
constexpr int kWNT = 256;
template <typename T>
__global__ void __launch_bounds__(kWNT)
encode_weights_kernel(int64_t cout, int64_t cin, int64_t pitch, bool transpose, const T* __restrict__ w,
                      uint8_t* __restrict__ codes, float* __restrict__ scales) {
  __shared__ uint8_t tile[kBlock][kBlock + 4];
  __shared__ uint32_t most[kWNT / 32];
  const int64_t o0 = (int64_t)blockIdx.y * kBlock, c0 = (int64_t)blockIdx.x * kBlock;
  // the source's rows: outputs, or (transposed) channels
  const int64_t r0 = transpose ? c0 : o0, q0 = transpose ? o0 : c0;
  const int64_t nr = transpose ? cin : cout, nq = transpose ? cout : cin;
  uint32_t m = 0;
  for (int i = threadIdx.x; i < kBlock * kBlock; i += kWNT) {
    const int64_t r = r0 + i / kBlock, q = q0 + i % kBlock;
    if (r < nr && q < nq) m = max(m, abs_bits(ld(w + r * nq + q)));
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = m;
  __syncthreads();
  m = 0;
#pragma unroll
  for (int k = 0; k < kWNT / 32; ++k) m = max(m, most[k]);
  float inv;
  const float s = scale_of<kSrcE4M3>(m, &inv);
  for (int i = threadIdx.x; i < kBlock * kBlock; i += kWNT) {
    const int a = i / kBlock, b = i % kBlock;
    const int64_t r = r0 + a, q = q0 + b;
    const uint8_t v = r < nr && q < nq ? encode1<kSrcE4M3>(ld(w + r * nq + q), inv) : 0;
    tile[transpose ? b : a][transpose ? a : b] = v;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kBlock * kBlock; i += kWNT) {
    const int a = i / kBlock, b = i % kBlock;
    if (o0 + a < cout) codes[(o0 + a) * pitch + c0 + b] = tile[a][b];
  }
  if (threadIdx.x == 0) scales[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = s;
}

// ---- aligned copy of codes -----------------------------------------------------

// Rows of cin bytes to rows of pitch bytes, zeros behind them; 16 bytes a
// thread, put together from the aligned words that hold them. Words that reach
// over an end of the tensor are read byte by byte.
__global__ void __launch_bounds__(256)
align_codes_kernel(int64_t rows, int cin, int64_t pitch, FastDiv d_vecs, const uint8_t* __restrict__ x, uint8_t* __restrict__ out) {
  dependents_may_start();
  const uint64_t total = (uint64_t)rows * (uint64_t)(pitch / 16);
  const uint8_t* const end = x + rows * cin;
  for (uint64_t i = blockIdx.x * (uint64_t)256 + threadIdx.x; i < total; i += (uint64_t)gridDim.x * 256) {
    int64_t r;
    int c;
    if (total < (uint64_t(1) << 32)) {
      uint32_t q;
      c = (int)d_vecs.divmod((uint32_t)i, q) * 16;
      r = q;
    } else {
      r = (int64_t)(i / (uint64_t)d_vecs.d);
      c = (int)(i - (uint64_t)r * d_vecs.d) * 16;
    }
    const uint8_t* p = x + r * cin + c;
    const int off = (int)(reinterpret_cast<uintptr_t>(p) & 3);
    const uint8_t* w0 = p - off;
    uint32_t v[4];
    if (c < cin && w0 >= x && w0 + 20 <= end) {
      uint32_t w[5];
#pragma unroll
      for (int k = 0; k < 5; ++k) w[k] = __ldg(reinterpret_cast<const uint32_t*>(w0) + k);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = __funnelshift_r(w[k], w[k + 1], 8 * off);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int left = cin - c - 4 * k;  // bytes of this word within the row
        v[k] = left >= 4 ? v[k] : left <= 0 ? 0 : v[k] & (0xffffffffu >> (32 - 8 * left));
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[k] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + 4 * k + e < cin) v[k] |= (uint32_t)__ldg(p + 4 * k + e) << (8 * e);
      }
    }
    *reinterpret_cast<uint4*>(out + r * pitch + c) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// ---- codes at any byte ------------------------------------------------------------

// 32 outputs x 8 pixels a block, one sum per thread; a block of channels of
// both at a time in shared memory, as values.
constexpr int kGO = 32, kGP = 8;
template <typename T>
__global__ void __launch_bounds__(kGO * kGP)
any_kernel(Pw g, int64_t ptiles, const uint8_t* __restrict__ x, const float* __restrict__ sx,
           const uint8_t* __restrict__ w, const float* __restrict__ sw, const T* __restrict__ bias, T* __restrict__ y) {
  __shared__ float xs[kGP][kBlock], ws[kGO][kBlock + 1];
  const int o = threadIdx.x % kGO, p = threadIdx.x / kGO;
  const int oo = blockIdx.x * kGO + o;
  for (int64_t pt = blockIdx.y; pt < ptiles; pt += gridDim.y) {
    const int64_t pp = pt * kGP + p;
    float acc = 0.f;
    for (int b = 0; b < g.nkb; ++b) {
      __syncthreads();
      for (int i = threadIdx.x; i < kGP * kBlock; i += kGO * kGP) {
        const int64_t r = pt * kGP + i / kBlock;
        const int c = b * kBlock + i % kBlock;
        xs[i / kBlock][i % kBlock] = r < g.rows && c < g.cin ? code1<kSrcE4M3>(__ldg(x + r * g.cin + c)) : 0.f;
      }
      for (int i = threadIdx.x; i < kGO * kBlock; i += kGO * kGP) {
        const int r = blockIdx.x * kGO + i / kBlock, c = b * kBlock + i % kBlock;
        ws[i / kBlock][i % kBlock] = r < g.cout && c < g.cin ? code1<kSrcE4M3>(__ldg(w + r * g.pitch + c)) : 0.f;
      }
      __syncthreads();
      if (pp < g.rows && oo < g.cout) {
        float d = 0.f;
        for (int c = 0; c < kBlock; ++c) d = fmaf(xs[p][c], ws[o][c], d);
        acc = fmaf(d, __fmul_rn(sx[pp * g.nkb + b], sw[(int64_t)(oo / kBlock) * g.nkb + b]), acc);
      }
    }
    if (pp < g.rows && oo < g.cout) {
      float v = bias ? acc + ld(bias + oo) : acc;
      norm::act_v<1>(g.act, &v);
      y[pp * g.ys + g.yo + oo] = from_f<T>(v);
    }
  }
}

template <typename T>
cudaError_t any(const Pw& g, const uint8_t* x, const float* sx, const uint8_t* w, const float* sw, const T* bias, T* y,
                cudaStream_t s) {
  const int64_t pt = (g.rows + kGP - 1) / kGP;
  any_kernel<T><<<dim3((g.cout + kGO - 1) / kGO, (unsigned)(pt < 65535 ? pt : 65535)), kGO * kGP, 0, s>>>(
      g, pt, x, sx, w, sw, bias, y);
  return cudaGetLastError();
}

}  // namespace

cudaError_t encode_weights(int64_t cout, int64_t cin, bool transpose, int dtype, const void* w, uint8_t* codes,
                           float* scales, cudaStream_t s) {
  const dim3 grid((unsigned)((cin + kBlock - 1) / kBlock), (unsigned)((cout + kBlock - 1) / kBlock));
  DWCONV_DISPATCH_DTYPE(dtype, T, encode_weights_kernel<T><<<grid, kWNT, 0, s>>>(cout, cin, pitch_of(cin), transpose,
                                                                                 (const T*)w, codes, scales));
  return cudaGetLastError();
}

size_t workspace_bytes(const Pw& g) { return g.cin % 16 == 0 ? 0 : (size_t)g.rows * (size_t)g.pitch; }

cudaError_t run(const Pw& g, const uint8_t* x, const float* sx, const uint8_t* w, const float* sw, const void* bias,
                void* y, void* ws, cudaStream_t s) {
  if (g.rows == 0) return cudaSuccess;
  cudaError_t e = cudaErrorNotSupported;
  const bool w16 = reinterpret_cast<uintptr_t>(w) % 16 == 0;
  if (w16 && g.cin % 16 != 0) {
    const int64_t total = g.rows * (g.pitch / 16), blocks = (total + 255) / 256;
    align_codes_kernel<<<(unsigned)(blocks < 152 * 8 ? blocks : 152 * 8), 256, 0, s>>>(g.rows, g.cin, g.pitch, FastDiv((uint32_t)(g.pitch / 16)), x, (uint8_t*)ws);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = run_tc(g, g.pitch, (const uint8_t*)ws, true, sx, w, sw, bias, y, s);
  } else if (w16 && reinterpret_cast<uintptr_t>(x) % 16 == 0) {
    e = run_tc(g, g.cin, x, false, sx, w, sw, bias, y, s);
  }
  if (e != cudaErrorNotSupported) return e;
  DWCONV_DISPATCH_DTYPE(g.dtype, T, e = any<T>(g, x, sx, w, sw, (const T*)bias, (T*)y, s));
  return e;
}

}  // namespace pw8
}  // namespace dwconv
