// RMS norm, backward (formulas of the forward in rms.cu):
//
//   t = gy * gamma,  gx = r * (t - h * r^2 * sum_c (t * h) / C) + gres
//   ggamma[c] = sum over rows of gy * (h * r)
//
// gres is the gradient that reaches h past the norm: gx is then the gradient
// of both x and the residual.
//
// Blocks walk over rows. A thread holds the same channels of every row that
// it meets, so its share of ggamma stays in registers from row to row; the
// next row's vectors are on their way while one is worked on. Row sums go
// through shuffles and, for rows of several warps, one exchange in shared
// memory (two buffers in turn: one barrier per row). The blocks' shares go to
// the workspace and a second launch adds them in a fixed order. Rows of more
// channels than 512 threads hold are read twice by one block, and a kernel of
// its own takes their ggamma, down the columns.
//
// Bound by memory: h, gy (and gres) read once, gx written once.
#include "rms.cuh"

namespace dwconv {
namespace rms {
namespace {

struct BGeom {
  int64_t rows, xs, xo, ys, yo;
  int C, nvec, tpr, log_tpr;
  float inv_c;
};

template <int NT>
__device__ __forceinline__ float row_sum(float s, int tpr, float* part) {
  const int tid = threadIdx.x, lane = tid & 31;
  const int W = tpr < 32 ? tpr : 32;
  for (int o = W >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (tpr > 32) {
    if (lane == 0) part[tid >> 5] = s;
    __syncthreads();
    const int nw = tpr >> 5, w0 = (tid >> 5) & ~(nw - 1);
    s = lane < nw ? part[w0 + lane] : 0.f;
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  }
  return s;
}

// AHEAD: the next row's vectors are loaded before this one is worked on.
template <typename T, int V, int NI, int NT, bool AHEAD>
__global__ void __launch_bounds__(NT)
bwd_kernel(BGeom g, const T* __restrict__ h, const T* __restrict__ gy, const T* __restrict__ gamma,
           const float* __restrict__ rstd, const T* gres, T* gx, float* __restrict__ shares) {
  typedef typename Raw<T, V>::type R;
  __shared__ float part[2][NT / 32];
  extern __shared__ float cols[];  // [C], where a block's rows are joined
  const int tid = threadIdx.x;
  const int in_row = tid & (g.tpr - 1);
  const int W = g.tpr < 32 ? g.tpr : 32;
  const int first = (in_row & ~(W - 1)) * NI + (in_row & (W - 1));
  const int rpb = NT >> g.log_tpr, grp = tid >> g.log_tpr;
  const int64_t step = (int64_t)gridDim.x * rpb;
  dependents_may_start();

  R gv[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i)
    if (gamma && first + i * W < g.nvec) gv[i] = *reinterpret_cast<const R*>(gamma + (int64_t)(first + i * W) * V);
  float acc[NI][V];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) acc[i][e] = 0.f;

  struct Row {
    R h[NI], gy[NI], gr[NI];
    float r;
  };
  auto fetch = [&](Row& q, int64_t row) {
    if (row >= g.rows) return;
    const T* hp = h + row * g.xs + g.xo;
    const T* yp = gy + row * g.ys + g.yo;
    const T* rp = gres ? gres + row * g.xs + g.xo : nullptr;
    q.r = __ldg(rstd + row);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int v = first + i * W;
      if (v >= g.nvec) continue;
      q.h[i] = *reinterpret_cast<const R*>(hp + (int64_t)v * V);
      q.gy[i] = *reinterpret_cast<const R*>(yp + (int64_t)v * V);
      if (rp && gx) q.gr[i] = *reinterpret_cast<const R*>(rp + (int64_t)v * V);
    }
  };
  int flip = 0;
  Row now, next;
  const int64_t row0 = (int64_t)blockIdx.x * rpb;
  if (AHEAD) fetch(now, row0 + grp);
  for (int64_t base = row0; base < g.rows; base += step, flip ^= 1) {  // the same for all threads of a block
    const int64_t row = base + grp;
    const bool live = row < g.rows;
    if (AHEAD) fetch(next, row + step);
    else fetch(now, row);
    const float r = live ? now.r : 0.f;
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (!live || first + i * W >= g.nvec) continue;
      float a[V], b[V], gm[V];
      widen<T, V>(now.h[i], a);
      widen<T, V>(now.gy[i], b);
      if (gamma) widen<T, V>(gv[i], gm);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        acc[i][e] = fmaf(b[e], __fmul_rn(a[e], r), acc[i][e]);
        const float t = gamma ? b[e] * gm[e] : b[e];
        (e & 1 ? s1 : s0) = fmaf(t, a[e], e & 1 ? s1 : s0);
      }
    }
    if (gx) {
      // (t . h) r / C: the mean of t * (h r)
      const float c1 = __fmul_rn(__fmul_rn(row_sum<NT>(s0 + s1, g.tpr, part[flip]), r), g.inv_c);
      T* op = gx + row * g.xs + g.xo;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int v = first + i * W;
        if (!live || v >= g.nvec) continue;
        float a[V], b[V], gm[V], q[V], o[V];
        widen<T, V>(now.h[i], a);
        widen<T, V>(now.gy[i], b);
        if (gamma) widen<T, V>(gv[i], gm);
        if (gres) widen<T, V>(now.gr[i], q);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float t = gamma ? b[e] * gm[e] : b[e];
          o[e] = fmaf(-__fmul_rn(a[e], r), c1, t);
          o[e] = gres ? fmaf(o[e], r, q[e]) : __fmul_rn(o[e], r);
        }
        *reinterpret_cast<R*>(op + (int64_t)v * V) = narrow<T, V>(o);
      }
    }
    if (AHEAD) now = next;
  }
  if (!shares) return;
  // the block's rows in order, then one line of the workspace
  for (int k = 0; k < rpb; ++k) {
    if (grp == k) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (first + i * W >= g.nvec) continue;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int c = (first + i * W) * V + e;
          const float u = k ? cols[c] + acc[i][e] : acc[i][e];
          if (k == rpb - 1) shares[(int64_t)blockIdx.x * g.C + c] = u;
          else cols[c] = u;
        }
      }
    }
    if (k + 1 < rpb) __syncthreads();
  }
}

// Rows too wide for the registers: one block per row, read twice.
constexpr int kWideNT = 512;
template <typename T>
__global__ void __launch_bounds__(kWideNT)
bwd_wide_kernel(BGeom g, const T* __restrict__ h, const T* __restrict__ gy, const T* __restrict__ gamma,
                const float* __restrict__ rstd, const T* gres, T* gx) {
  __shared__ float part[kWideNT / 32];
  for (int64_t row = blockIdx.x; row < g.rows; row += gridDim.x) {
    const T* hp = h + row * g.xs + g.xo;
    const T* yp = gy + row * g.ys + g.yo;
    const T* rp = gres ? gres + row * g.xs + g.xo : nullptr;
    T* op = gx + row * g.xs + g.xo;
    const float r = __ldg(rstd + row);
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c0 = threadIdx.x; c0 < g.C; c0 += 4 * kWideNT) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = c0 + k * kWideNT;
        if (c < g.C) s[k] = fmaf(gamma ? ld(yp + c) * ld(gamma + c) : ld(yp + c), ld(hp + c), s[k]);
      }
    }
    const float c1 = __fmul_rn(__fmul_rn(row_sum<kWideNT>((s[0] + s[1]) + (s[2] + s[3]), kWideNT, part), r), g.inv_c);
    for (int c = threadIdx.x; c < g.C; c += kWideNT) {
      const float t = gamma ? ld(yp + c) * ld(gamma + c) : ld(yp + c);
      const float o = fmaf(-__fmul_rn(ld(hp + c), r), c1, t);
      op[c] = from_f<T>(rp ? fmaf(o, r, ld_rw(rp + c)) : __fmul_rn(o, r));
    }
    __syncthreads();  // part is written again for the next row
  }
}

// ggamma of rows too wide: a thread per column and share of the rows.
template <typename T>
__global__ void __launch_bounds__(256)
columns_kernel(BGeom g, int chunks, const T* __restrict__ h, const T* __restrict__ gy, const float* __restrict__ rstd,
               float* __restrict__ shares) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  const int64_t r0 = g.rows * blockIdx.y / chunks, r1 = g.rows * (blockIdx.y + 1) / chunks;
  dependents_may_start();
  if (c >= g.C) return;
  float acc = 0.f;
  for (int64_t row = r0; row < r1; ++row)
    acc = fmaf(ld(gy + row * g.ys + g.yo + c), __fmul_rn(ld(h + row * g.xs + g.xo + c), __ldg(rstd + row)), acc);
  shares[(int64_t)blockIdx.y * g.C + c] = acc;
}

// ggamma[c] = the shares' sum, in a fixed order: 8 columns and 64 row lanes a
// block, each lane every 64th share, then the lanes in a tree.
constexpr int kJoinCols = 8, kJoinLanes = 64;
template <typename T>
__global__ void __launch_bounds__(kJoinCols * kJoinLanes)
join_kernel(int C, int n, const float* __restrict__ shares, T* __restrict__ ggamma) {
  __shared__ float sm[kJoinLanes][kJoinCols + 1];
  const int k = threadIdx.x % kJoinCols, l = threadIdx.x / kJoinCols;
  const int c = blockIdx.x * kJoinCols + k;
  wait_for_previous();
  float a = 0.f;
  if (c < C) {
#pragma unroll 8
    for (int b = l; b < n; b += kJoinLanes) a += shares[(int64_t)b * C + c];
  }
  sm[l][k] = a;
  __syncthreads();
  for (int o = kJoinLanes / 2; o > 0; o >>= 1) {
    if (l < o) sm[l][k] += sm[l + o][k];
    __syncthreads();
  }
  if (l == 0 && c < C) ggamma[c] = from_f<T>(sm[0][k]);
}

template <typename T>
__global__ void zero_kernel(int C, T* ggamma) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c < C) ggamma[c] = from_f<T>(0.f);
}

// 16 channels at most per thread (their shares of ggamma are registers), and
// at most 512 threads to a row.
constexpr int kHeld = 16;
Lay lay(const Rms& g, int V) {
  Lay l{};
  l.v = V;
  const int64_t nvec = g.C / V;
  l.ni = V == 1 ? kHeld : nvec > 128 ? kHeld / V : 1;
  const int64_t need = (nvec + l.ni - 1) / l.ni;
  l.tpr = pow2_at_least(need);
  if (l.tpr < 4) l.tpr = 4;
  l.nt = l.tpr > 256 ? 512 : 256;
  if (l.tpr > 512) l.tpr = 512;
  l.segs = (int)((need + l.tpr - 1) / l.tpr);
  return l;
}

// Blocks that walk over the rows: as many as stay on the GPU at once, more
// where a thread would add up over 4096 rows.
constexpr int64_t kBlocks = 152 * 4, kMostRows = 4096;
int64_t blocks_of(const Rms& g, const Lay& l) {
  const int64_t rpb = l.nt / l.tpr, all = (g.rows + rpb - 1) / rpb;
  int64_t n = l.nt == 512 ? kBlocks / 2 : kBlocks;
  if ((all + n - 1) / n > kMostRows) n = (all + kMostRows - 1) / kMostRows;
  return all < n ? all : n;
}
int64_t chunks_of(const Rms& g) {
  const int64_t n = (g.rows + 63) / 64;
  return n < 1 ? 1 : n < 256 ? n : g.rows / kMostRows > 256 ? (g.rows / kMostRows < 65535 ? g.rows / kMostRows : 65535) : 256;
}

int64_t shares_of(const Rms& g, int V) {
  const Lay l = lay(g, V);
  return l.segs == 1 ? blocks_of(g, l) : chunks_of(g);
}

template <typename T, int V, int NI>
cudaError_t launch(const BGeom& f, const Lay& l, int64_t blocks, const T* h, const T* gy, const T* gamma,
                   const float* rstd, const T* gres, T* gx, float* ws, cudaStream_t s) {
  const size_t smem = ws && l.nt > l.tpr ? (size_t)f.C * 4 : 0;
  if (l.nt == 256) bwd_kernel<T, V, NI, 256, true><<<(unsigned)blocks, 256, smem, s>>>(f, h, gy, gamma, rstd, gres, gx, ws);
  else bwd_kernel<T, V, NI, 512, false><<<(unsigned)blocks, 512, smem, s>>>(f, h, gy, gamma, rstd, gres, gx, ws);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run(const Rms& g, const T* h, const T* gy, const T* gamma, const float* rstd, const T* gres, T* gx,
                T* ggamma, float* ws, cudaStream_t s) {
  constexpr int VEC = Vec<T>::n;
  cudaError_t e = cudaSuccess;
  if (g.rows == 0) {
    if (ggamma) zero_kernel<T><<<(g.C + 255) / 256, 256, 0, s>>>(g.C, ggamma);
    return cudaGetLastError();
  }
  if (!ggamma) ws = nullptr;
  const int V = vec_ok(g, VEC, on16(h) && on16(gy) && on16(gamma) && on16(gres) && on16(gx), nullptr) ? VEC : 1;
  const Lay l = lay(g, V);
  BGeom f{};
  f.rows = g.rows;
  f.xs = g.xs; f.xo = g.xo; f.ys = g.ys; f.yo = g.yo;
  f.C = g.C;
  f.nvec = g.C / V;
  f.tpr = l.tpr;
  while ((1 << f.log_tpr) < l.tpr) ++f.log_tpr;
  f.inv_c = 1.f / (float)g.C;
  int64_t n;
  if (l.segs > 1) {
    n = chunks_of(g);
    if (gx) {
      bwd_wide_kernel<T><<<(unsigned)(g.rows < 152 * 8 ? g.rows : 152 * 8), kWideNT, 0, s>>>(f, h, gy, gamma, rstd, gres, gx);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (ws) columns_kernel<T><<<dim3((g.C + 255) / 256, (unsigned)n), 256, 0, s>>>(f, (int)n, h, gy, rstd, ws);
    e = cudaGetLastError();
  } else {
    n = blocks_of(g, l);
    if (V == 1) e = launch<T, 1, kHeld>(f, l, n, h, gy, gamma, rstd, gres, gx, ws, s);
    else if (l.ni == 1) e = launch<T, VEC, 1>(f, l, n, h, gy, gamma, rstd, gres, gx, ws, s);
    else e = launch<T, VEC, kHeld / VEC>(f, l, n, h, gy, gamma, rstd, gres, gx, ws, s);
  }
  if (e != cudaSuccess || !ws) return e;
  return launch_dependent(join_kernel<T>, dim3((g.C + kJoinCols - 1) / kJoinCols), dim3(kJoinCols * kJoinLanes), 0, s, g.C,
                          (int)n, (const float*)ws, ggamma);
}

}  // namespace

const char* plan_name(const Rms& g, int pass) {
  if (pass == 0) return fwd_in_row(g) ? "row" : "wide";
  const int VEC = g.dtype == DWCONV_F32 ? 4 : 8;
  return lay(g, vec_ok(g, VEC, true, nullptr) ? VEC : 1).segs == 1 ? "row" : "wide";
}

size_t bwd_workspace_bytes(const Rms& g) {
  const int VEC = g.dtype == DWCONV_F32 ? 4 : 8;
  int64_t n = shares_of(g, 1);  // pointers off 16 bytes take elements one by one
  if (g.C % VEC == 0) {
    const int64_t m = shares_of(g, VEC);
    if (m > n) n = m;
  }
  return (size_t)(n < 1 ? 1 : n) * g.C * sizeof(float);
}

cudaError_t bwd(const Rms& g, const void* h, const void* gy, const void* gamma, const float* rstd, const void* gres,
                void* gx, void* ggamma, float* ws, cudaStream_t s) {
  cudaError_t e = cudaErrorInvalidValue;
  DWCONV_DISPATCH_DTYPE(g.dtype, T, e = run<T>(g, (const T*)h, (const T*)gy, (const T*)gamma, rstd, (const T*)gres,
                                               (T*)gx, (T*)ggamma, ws, s));
  return e;
}

}  // namespace rms
}  // namespace dwconv
