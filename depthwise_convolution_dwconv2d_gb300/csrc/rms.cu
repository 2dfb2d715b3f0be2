// RMS norm over the channels of a row (channels-last), forward:
//
//   h = x + residual, rounded to the storage type (h = x without a residual)
//   r = 1 / sqrt(sum_c h^2 / C + eps),  y = (h * r) * gamma
//
// and y is rounded once, to the storage type, to 8-bit codes with one scale
// per block of channels (act8.cuh), or to both. The norm is taken of h as
// stored, so that the backward, which reads h, finds the same values; sums
// and statistics are fp32.
//
// One pass: a row is read once into the registers of its threads, as stored
// (h needs no more bits), its sum of squares goes through shuffles and, for
// rows of several warps, one exchange in shared memory; the codes' maxima are
// shuffles of the lanes that hold a block. Rows of more channels than 1024
// threads hold are read twice, in spans.
//
// Bound by memory: 4 to 6 operations per element against 2 to 7 bytes.
#include "rms.cuh"

namespace dwconv {
namespace rms {
namespace {

struct FGeom {
  int64_t rows, xs, xo, ys, yo;
  int C, nvec;      // channels and vectors of a row
  int tpr, log_tpr;
  int segs;
  float eps, inv_c;
};

template <typename T, int V, int NI, int Q, int NT>
__global__ void __launch_bounds__(NT)
fwd_kernel(FGeom g, const T* x, const T* res, const T* __restrict__ gamma, T* h, T* y,
           float* rstd, Act8 t) {
  typedef typename Raw<T, V>::type R;
  __shared__ float part[NT / 32];
  const int tid = threadIdx.x, lane = tid & 31;
  const int in_row = tid & (g.tpr - 1);
  const int W = g.tpr < 32 ? g.tpr : 32;
  const int first = (in_row & ~(W - 1)) * NI + (in_row & (W - 1));  // vector of item 0; item i is i * W further
  const int span = g.tpr * NI;
  const int64_t row = (int64_t)blockIdx.x * (NT >> g.log_tpr) + (tid >> g.log_tpr);
  const bool live = row < g.rows;
  const T* xr = x + row * g.xs + g.xo;
  const T* rr = res + (res ? row * g.xs + g.xo : 0);
  T* hr = h + (h ? row * g.xs + g.xo : 0);

  R hv[NI], gv[NI];
  auto load_h = [&](int seg, bool again) {
    R rv[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int v = seg * span + first + i * W;
      if (live && v < g.nvec) {
        // the second read of a row takes h where it was stored: x or the residual may be the same memory
        hv[i] = *reinterpret_cast<const R*>((again && h ? hr : xr) + (int64_t)v * V);
        if (res && !(again && h)) rv[i] = *reinterpret_cast<const R*>(rr + (int64_t)v * V);
      }
    }
    if (res && !(again && h)) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int v = seg * span + first + i * W;
        if (live && v < g.nvec) {
          float a[V], b[V];
          widen<T, V>(hv[i], a);
          widen<T, V>(rv[i], b);
#pragma unroll
          for (int e = 0; e < V; ++e) a[e] += b[e];
          hv[i] = narrow<T, V>(a);
        }
      }
    }
    if (h && !again) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int v = seg * span + first + i * W;
        if (live && v < g.nvec) *reinterpret_cast<R*>(hr + (int64_t)v * V) = hv[i];
      }
    }
  };
  auto load_gamma = [&](int seg) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int v = seg * span + first + i * W;
      if (gamma && v < g.nvec) gv[i] = *reinterpret_cast<const R*>(gamma + (int64_t)v * V);
    }
  };

  float ss = 0.f;
  for (int seg = 0; seg < g.segs; ++seg) {
    if (g.segs == 1) load_gamma(0);
    load_h(seg, false);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int v = seg * span + first + i * W;
      if (live && v < g.nvec) {
        float a[V];
        widen<T, V>(hv[i], a);
#pragma unroll
        for (int e = 0; e < V; ++e) (e & 1 ? s1 : s0) = fmaf(a[e], a[e], e & 1 ? s1 : s0);
      }
    }
    ss += s0 + s1;
  }
  for (int o = W >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (g.tpr > 32) {
    if (lane == 0) part[tid >> 5] = ss;
    __syncthreads();
    const int nw = g.tpr >> 5, w0 = (tid >> 5) & ~(nw - 1);
    ss = lane < nw ? part[w0 + lane] : 0.f;
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  }
  const float r = __frsqrt_rn(fmaf(ss, g.inv_c, g.eps));
  if (live && in_row == 0 && rstd) rstd[row] = r;

  T* yr = y + (y ? row * g.ys + g.yo : 0);
  for (int seg = 0; seg < g.segs; ++seg) {
    if (g.segs > 1) {
      load_gamma(seg);
      load_h(seg, true);
    }
    float f[NI][V];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int v = seg * span + first + i * W;
      const bool on = live && v < g.nvec;
      float gm[V];
      if (on) {
        widen<T, V>(hv[i], f[i]);
        if (gamma) widen<T, V>(gv[i], gm);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        f[i][e] = on ? __fmul_rn(f[i][e], r) : 0.f;
        if (on && gamma) f[i][e] = __fmul_rn(f[i][e], gm[e]);
      }
      if (y && on) *reinterpret_cast<R*>(yr + (int64_t)v * V) = narrow<T, V>(f[i]);
    }
    if constexpr (Q != kSrcFull) {
      const int block = 1 << t.shift;
      uint32_t m[NI];
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        m[i] = 0;
#pragma unroll
        for (int e = 0; e < V; ++e) m[i] = max(m[i], abs_bits(f[i][e]));
      }
      int lanes = block / V;  // a block's lanes, or all of the row's
      if (lanes > W) {
        // several items of a thread are of one block (V == 1, or a row that ends within the block)
        int ipb = lanes / W;
        if (ipb > NI) ipb = NI;
#pragma unroll
        for (int o = 1; o < NI; o <<= 1) {
          if (o < ipb) {
            uint32_t u[NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) u[i] = max(m[i], m[i ^ o]);
#pragma unroll
            for (int i = 0; i < NI; ++i) m[i] = u[i];
          }
        }
        lanes = W;
      }
      for (int o = lanes >> 1; o > 0; o >>= 1) {
#pragma unroll
        for (int i = 0; i < NI; ++i) m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int v = seg * span + first + i * W;
        if (!live || v >= g.nvec) continue;
        const int c = v * V;
        float inv;
        const float s = scale_of<Q>(m[i], &inv);
        uint8_t* q = t.codes + row * g.C + c;
        if constexpr (V == 8) {
          *reinterpret_cast<uint2*>(q) = make_uint2(encode4<Q>(f[i][0], f[i][1], f[i][2], f[i][3], inv),
                                                    encode4<Q>(f[i][4], f[i][5], f[i][6], f[i][7], inv));
        } else if constexpr (V == 4) {
          *reinterpret_cast<uint32_t*>(q) = encode4<Q>(f[i][0], f[i][1], f[i][2], f[i][3], inv);
        } else {
          *q = encode1<Q>(f[i][0], inv);
        }
        if ((c & (block - 1)) == 0) t.scales[row * t.nblk + (c >> t.shift)] = s;
      }
    }
  }
}

// Vectors per thread: one while all rows together are less than a wave of
// threads (latency counts), else two, or four where 256 threads then hold a
// row. Elements one by one are taken eight to a thread.
Lay lay(const Rms& g, int V) {
  Lay l{};
  l.v = V;
  const int64_t nvec = g.C / V;
  if (V == 1) {
    l.ni = 8;
  } else {
    const bool wave = g.rows * nvec > 152 * 2048;
    l.ni = nvec > 1024 ? 2 : !wave || nvec < 64 ? 1 : nvec < 128 ? 2 : 4;
  }
  const int64_t need = (nvec + l.ni - 1) / l.ni;
  l.tpr = pow2_at_least(need);
  if (l.tpr < 4) l.tpr = 4;
  if (l.tpr > 1024) l.tpr = 1024;
  l.nt = l.tpr > 256 ? l.tpr : 256;
  l.segs = (int)((need + l.tpr - 1) / l.tpr);
  return l;
}

template <typename T, int V, int NI, int Q>
cudaError_t launch(const Rms& g, const Lay& l, const T* x, const T* res, const T* gamma, T* h, T* y, float* rstd,
                   const Act8& t, cudaStream_t s) {
  FGeom f{};
  f.rows = g.rows;
  f.xs = g.xs; f.xo = g.xo; f.ys = g.ys; f.yo = g.yo;
  f.C = g.C;
  f.nvec = g.C / V;
  f.tpr = l.tpr;
  while ((1 << f.log_tpr) < l.tpr) ++f.log_tpr;
  f.segs = l.segs;
  f.eps = g.eps;
  f.inv_c = 1.f / (float)g.C;
  const int64_t rpb = l.nt / l.tpr, most = (int64_t(1) << 30);
  for (int64_t r = 0; r < g.rows; r += most * rpb) {
    f.rows = g.rows - r < most * rpb ? g.rows - r : most * rpb;
    const unsigned grid = (unsigned)((f.rows + rpb - 1) / rpb);
    Act8 u = t;
    if (Q != kSrcFull) {
      u.codes += r * g.C;
      u.scales += r * t.nblk;
    }
    const int64_t ox = r * g.xs, oy = r * g.ys;
    const T* r2 = res ? res + ox : nullptr;
    T* h2 = h ? h + ox : nullptr;
    T* y2 = y ? y + oy : nullptr;
    float* s2 = rstd ? rstd + r : nullptr;
    if (l.nt == 256) fwd_kernel<T, V, NI, Q, 256><<<grid, 256, 0, s>>>(f, x + ox, r2, gamma, h2, y2, s2, u);
    if constexpr (NI != 4) {
      if (l.nt == 512) fwd_kernel<T, V, NI, Q, 512><<<grid, 512, 0, s>>>(f, x + ox, r2, gamma, h2, y2, s2, u);
      if (l.nt == 1024) fwd_kernel<T, V, NI, Q, 1024><<<grid, 1024, 0, s>>>(f, x + ox, r2, gamma, h2, y2, s2, u);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T, int Q>
cudaError_t run(const Rms& g, const void* x, const void* res, const void* gamma, void* h, void* y, float* rstd,
                const Act8& t, cudaStream_t s) {
  constexpr int VEC = Vec<T>::n;
  const bool v = vec_ok(g, VEC, on16(x) && on16(res) && on16(gamma) && on16(h) && on16(y), Q != kSrcFull ? t.codes : nullptr);
  const Lay l = lay(g, v ? VEC : 1);
#define GO(V_, NI_) return launch<T, V_, NI_, Q>(g, l, (const T*)x, (const T*)res, (const T*)gamma, (T*)h, (T*)y, rstd, t, s)
  if (!v) GO(1, 8);
  if (l.ni == 1) GO(VEC, 1);
  if (l.ni == 2) GO(VEC, 2);
  GO(VEC, 4);
#undef GO
}

}  // namespace

bool fwd_in_row(const Rms& g) {
  const int VEC = g.dtype == DWCONV_F32 ? 4 : 8;
  return lay(g, vec_ok(g, VEC, true, nullptr) ? VEC : 1).segs == 1;
}

cudaError_t fwd(const Rms& g, const void* x, const void* residual, const void* gamma, void* h, void* y, float* rstd,
                const Act8& t, cudaStream_t s) {
  if (g.rows == 0) return cudaSuccess;
  cudaError_t e = cudaErrorInvalidValue;
  if (!t.codes) {
    DWCONV_DISPATCH_DTYPE(g.dtype, T, e = run<T, kSrcFull>(g, x, residual, gamma, h, y, rstd, t, s));
  } else if (t.src == kSrcI8) {
    DWCONV_DISPATCH_DTYPE(g.dtype, T, e = run<T, kSrcI8>(g, x, residual, gamma, h, y, rstd, t, s));
  } else {
    DWCONV_DISPATCH_DTYPE(g.dtype, T, e = run<T, kSrcE4M3>(g, x, residual, gamma, h, y, rstd, t, s));
  }
  return e;
}

}  // namespace rms
}  // namespace dwconv
