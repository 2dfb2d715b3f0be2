// RMS norm, backward (formulas of the forward in rms.cu):
//
//   t = gy * gamma,  gx = r * (t - h * r^2 * sum_c (t * h) / C) + gres
//   ggamma[c] = sum over rows of gy * (h * r)
//
// gres is the gradient that reaches h past the norm: gx is then the gradient
// of both x and the residual.
//
// Blocks walk over rows. A thread holds the same channels of every row that
// it meets (rows that begin off 16 bytes too: it steps over rows that begin
// alike, rms.cuh), so its share of ggamma stays in registers from row to row;
// the next row's vectors are on their way while one is worked on. Row sums go
// through shuffles and, for rows of several warps, one exchange in shared
// memory (two buffers in turn: one barrier per row). The blocks' shares go to
// the workspace and a second launch adds them in a fixed order. Rows of more
// channels than 512 threads hold, and tensors that do not begin alike, are
// read element by element, twice, by one block, and a kernel of its own takes
// their ggamma, down the columns.
//
// Bound by memory: h, gy (and gres) read once, gx written once.
#include "rms.cuh"

namespace dwconv {
namespace rms {
namespace {

struct BGeom {
  int64_t rows, xs, xo, ys, yo;
  int C, tpr, log_tpr;
  float inv_c;
};

// AHEAD: the next row's vectors are loaded before this one is worked on.
template <typename T, int V, int NI, int NT, bool AHEAD, bool RAG>
__global__ void __launch_bounds__(NT, NT == 256 ? (NI == 1 ? 3 : 2) : 1)
bwd_kernel(BGeom g, const T* __restrict__ h, const T* __restrict__ gy, const T* __restrict__ gamma,
           const float* __restrict__ rstd, const T* gres, T* gx, float* __restrict__ shares) {
  typedef typename Raw<T, V>::type R;
  constexpr int P = V / 2;
  __shared__ float part[2][NT / 32];
  extern __shared__ float cols[];  // [C], where a block's rows are joined
  const int tid = threadIdx.x;
  const int in_row = tid & (g.tpr - 1);
  const int W = NI > 1 || g.tpr >= 32 ? 32 : g.tpr;  // rows of fewer than 32 lanes have one vector a lane
  const int first = (in_row & ~(W - 1)) * NI + (in_row & (W - 1));
  const int rpb = NT >> g.log_tpr, grp = tid >> g.log_tpr;
  const int64_t step = (int64_t)gridDim.x * rpb;  // RAG: a multiple of 8
  int64_t row = (int64_t)blockIdx.x * rpb + grp;
  const int ph = RAG ? phase_of(h + row * g.xs + g.xo) : 0;
  const int nvec = (g.C + ph + V - 1) / V;
  const int c0 = first * V - ph;  // first channel of item 0; item i is 32 V further
  const int64_t xstep = step * g.xs, ystep = step * g.ys;
  const T* hp = h + row * g.xs + g.xo;
  const T* yp = gy + row * g.ys + g.yo;
  const T* rp = gres + (gres ? row * g.xs + g.xo : 0);
  T* op = gx + (gx ? row * g.xs + g.xo : 0);
  dependents_may_start();

  f32x2 gm[NI][P], acc[NI][P];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
#pragma unroll
    for (int e = 0; e < P; ++e) {
      gm[i][e] = both(1.f);
      acc[i][e] = 0ull;
    }
    if (gamma && first + i * W < nvec)
      pairs_of<T, V>(RAG ? load_part<T, V>(gamma, c0 + i * W * V, g.C) : load_vec<T, V, false>(gamma, c0 + i * W * V, g.C), gm[i]);
  }

  R nh[NI], ny[NI], nr[NI];
  float next_r = 0.f;
  auto fetch = [&](int64_t at) {  // the row that the pointers are at
    next_r = 0.f;
    if (at >= g.rows) return;
    next_r = __ldg(rstd + at);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (first + i * W >= nvec) continue;
      nh[i] = load_vec<T, V, RAG>(hp, c0 + i * W * V, g.C);
      ny[i] = load_vec<T, V, RAG>(yp, c0 + i * W * V, g.C);
      if (gres && gx) nr[i] = load_vec<T, V, RAG>(rp, c0 + i * W * V, g.C);
    }
  };
  int flip = 0;
  if (AHEAD) fetch(row);
  for (int64_t base = (int64_t)blockIdx.x * rpb; base < g.rows; base += step, row += step, flip ^= 1) {  // the same for all threads of a block
    const bool live = row < g.rows;
    if (!AHEAD) fetch(row);
    const float r = next_r;
    R gr[NI];
    f32x2 s2 = 0ull, xh[NI][P], t[NI][P];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (!live || first + i * W >= nvec) continue;
      pairs_of<T, V>(nh[i], xh[i]);
      pairs_of<T, V>(ny[i], t[i]);
      if (gres) gr[i] = nr[i];
#pragma unroll
      for (int e = 0; e < P; ++e) {
        xh[i][e] = mul_f32x2(xh[i][e], both(r));
        acc[i][e] = fma2(t[i][e], xh[i][e], acc[i][e]);
        t[i][e] = mul_f32x2(t[i][e], gm[i][e]);
        s2 = fma2(t[i][e], xh[i][e], s2);
      }
    }
    hp += xstep;
    yp += ystep;
    rp += xstep;
    if (AHEAD) fetch(row + step);
    if (gx) {
      // the mean of t * (h r), negated
      const float c1 = -__fmul_rn(row_sum<NT>(sum2(s2), g.tpr, part[flip]), g.inv_c);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (!live || first + i * W >= nvec) continue;
        f32x2 q[P];
        if (gres) pairs_of<T, V>(gr[i], q);
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const f32x2 d = fma2(xh[i][e], both(c1), t[i][e]);
          q[e] = gres ? fma2(d, both(r), q[e]) : mul_f32x2(d, both(r));
        }
        store_vec<T, V, RAG>(op, c0 + i * W * V, g.C, vec_of<T, V>(q));
      }
      op += xstep;
    }
  }
  if (!shares) return;
  // the block's rows in order, then one line of the workspace
  float* mine = shares + (int64_t)blockIdx.x * g.C;
  for (int k = 0; k < rpb; ++k) {
    if (grp == k) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int c = c0 + i * W * V + e;
          if (c < 0 || c >= g.C) continue;
          float lo, hi;
          unpack_f32x2(acc[i][e / 2], lo, hi);
          const float u = k ? cols[c] + (e & 1 ? hi : lo) : (e & 1 ? hi : lo);
          if (k == rpb - 1) mine[c] = u;
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
Lay lay(const Rms& g, int V, bool ragged) {
  Lay l{};
  l.v = V;
  const int64_t nvec = ragged ? (g.C + 2 * V - 2) / V : g.C / V;
  l.ni = nvec <= 128 ? 1 : nvec <= 1024 ? 2 : kHeld / V;
  const int64_t need = (nvec + l.ni - 1) / l.ni;
  l.tpr = pow2_at_least(need);
  if (l.tpr < 4) l.tpr = 4;
  l.nt = l.tpr > 256 ? 512 : 256;
  if (l.tpr > 512) l.tpr = 512;
  l.segs = (int)((need + l.tpr - 1) / l.tpr);
  return l;
}

// Blocks that walk over the rows: as many as stay on the GPU at once, but four
// rows each at least where a row is of several warps (the shares are read
// again), more where a thread would add up over 4096 rows; rows in steps of 8.
constexpr int64_t kMostRows = 4096;
int64_t blocks_of(const Rms& g, const Lay& l) {
  const int64_t rpb = l.nt / l.tpr, all = (g.rows + rpb - 1) / rpb;
  int64_t n = 152 * (l.nt == 512 ? 1 : l.ni == 1 ? 3 : 2);
  if (l.tpr > 32 && n > (all + 3) / 4) n = (all + 3) / 4;
  if ((all + n - 1) / n > kMostRows) n = (all + kMostRows - 1) / kMostRows;
  if (all < n) n = all;
  while (n * rpb % 8) ++n;
  return n;
}
int64_t chunks_of(const Rms& g) {
  const int64_t n = (g.rows + 63) / 64;
  return n < 1 ? 1 : n < 256 ? n : g.rows / kMostRows > 256 ? (g.rows / kMostRows < 65535 ? g.rows / kMostRows : 65535) : 256;
}

template <typename T, int V, int NI, bool RAG>
cudaError_t launch(const BGeom& f, const Lay& l, int64_t blocks, const T* h, const T* gy, const T* gamma,
                   const float* rstd, const T* gres, T* gx, float* ws, cudaStream_t s) {
  const size_t smem = ws && l.nt > l.tpr ? (size_t)f.C * 4 : 0;
  if constexpr (NI <= 2) {
    if (l.nt == 256) {
      bwd_kernel<T, V, NI, 256, true, RAG><<<(unsigned)blocks, 256, smem, s>>>(f, h, gy, gamma, rstd, gres, gx, ws);
      return cudaGetLastError();
    }
  }
  bwd_kernel<T, V, NI, 512, false, RAG><<<(unsigned)blocks, 512, smem, s>>>(f, h, gy, gamma, rstd, gres, gx, ws);
  return cudaGetLastError();
}

template <typename T>
cudaError_t run(const Rms& g, const T* h, const T* gy, const T* gamma, const float* rstd, const T* gres, T* gx,
                T* ggamma, float* ws, cudaStream_t s) {
  constexpr int V = Vec<T>::n;
  cudaError_t e = cudaSuccess;
  if (g.rows == 0) {
    if (ggamma) zero_kernel<T><<<(g.C + 255) / 256, 256, 0, s>>>(g.C, ggamma);
    return cudaGetLastError();
  }
  if (!ggamma) ws = nullptr;
  const bool vec = rows_on16(g, V) && on16(h) && on16(gy) && on16(gamma) && on16(gres) && on16(gx);
  const Lay l = lay(g, V, !vec);
  BGeom f{};
  f.rows = g.rows;
  f.xs = g.xs; f.xo = g.xo; f.ys = g.ys; f.yo = g.yo;
  f.C = g.C;
  f.tpr = l.tpr;
  while ((1 << f.log_tpr) < l.tpr) ++f.log_tpr;
  f.inv_c = 1.f / (float)g.C;
  int64_t n;
  if (l.segs == 1 && (vec || (alike(h, gy) && alike(h, gres) && alike(h, gx) && rows_alike(g, V)))) {
    n = blocks_of(g, l);
    const auto go = vec ? (l.ni == 1 ? launch<T, V, 1, false> : l.ni == 2 ? launch<T, V, 2, false> : launch<T, V, kHeld / V, false>)
                        : (l.ni == 1 ? launch<T, V, 1, true> : l.ni == 2 ? launch<T, V, 2, true> : launch<T, V, kHeld / V, true>);
    e = go(f, l, n, h, gy, gamma, rstd, gres, gx, ws, s);
  } else {
    n = chunks_of(g);
    if (gx) {
      bwd_wide_kernel<T><<<(unsigned)(g.rows < 152 * 8 ? g.rows : 152 * 8), kWideNT, 0, s>>>(f, h, gy, gamma, rstd, gres, gx);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (ws) columns_kernel<T><<<dim3((g.C + 255) / 256, (unsigned)n), 256, 0, s>>>(f, (int)n, h, gy, rstd, ws);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || !ws) return e;
  return launch_dependent(join_kernel<T>, dim3((g.C + kJoinCols - 1) / kJoinCols), dim3(kJoinCols * kJoinLanes), 0, s, g.C,
                          (int)n, (const float*)ws, ggamma);
}

}  // namespace

const char* plan_name(const Rms& g, int pass) {
  if (pass == 0) return fwd_in_row(g) ? "row" : "wide";
  const int V = g.dtype == DWCONV_F32 ? 4 : 8;
  return lay(g, V, !rows_on16(g, V)).segs == 1 && rows_alike(g, V) ? "row" : "wide";
}

size_t bwd_workspace_bytes(const Rms& g) {
  const int V = g.dtype == DWCONV_F32 ? 4 : 8;
  int64_t n = chunks_of(g);  // pointers decide which kernel runs
  for (int ragged = 0; ragged < 2; ++ragged) {
    const Lay l = lay(g, V, ragged != 0);
    if (l.segs == 1 && n < blocks_of(g, l)) n = blocks_of(g, l);
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
