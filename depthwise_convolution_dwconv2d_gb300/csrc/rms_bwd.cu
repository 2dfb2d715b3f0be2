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
// their ggamma, down the columns. Both are laid out for wide rows (2000 x 30000
// bf16 with gres 354 us, 72 the floor); narrow ones that do not begin alike
// leave most of their threads idle (200704 x 128 bf16 560 us against 45).
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

// Rows are fetched by asynchronous copies, S rows ahead, into the thread's own
// slots of shared memory: no thread reads another's, so a thread waits for its
// own copies only. Three stages and three blocks per SM where a thread has one
// vector: four and four spill registers (200704 x 128 bf16 45 us against 35).
constexpr int stages_of(int ni) { return ni == 1 ? 3 : 2; }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ uint4 read16(uint32_t at) {
  uint4 u;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(at) : "memory");
  return u;
}

__device__ __forceinline__ void write16(uint32_t at, const uint4& u) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w) : "memory");
}

// GRES: gres and gx are given.
template <typename T, int V, int NI, int NT, bool RAG, bool GRES>
__global__ void __launch_bounds__(NT, NT == 256 ? (NI == 1 ? 3 : 2) : 1)
bwd_kernel(BGeom g, const T* __restrict__ h, const T* __restrict__ gy, const T* __restrict__ gamma,
           const float* __restrict__ rstd, const T* gres, T* gx, float* __restrict__ shares) {
  typedef typename Raw<T, V>::type R;
  constexpr int P = V / 2;
  constexpr int S = stages_of(NI);
  constexpr uint32_t kLine = NT * 16, kStage = 3 * NI * kLine;  // bytes of a vector of every thread, of a stage
  __shared__ float part[2][NT / 32];
  extern __shared__ __align__(16) unsigned char dyn[];
  const uint32_t slots = (uint32_t)__cvta_generic_to_shared(dyn) + threadIdx.x * 16;
  const int tid = threadIdx.x;
  const int in_row = tid & (g.tpr - 1);
  const int W = g.tpr < 32 ? g.tpr : 32;
  const int first = (in_row & ~(W - 1)) * NI + (in_row & (W - 1));
  const int rpb = NT >> g.log_tpr, grp = tid >> g.log_tpr;
  const int64_t step = (int64_t)gridDim.x * rpb;  // RAG: a multiple of 8
  const int64_t row = (int64_t)blockIdx.x * rpb + grp;
  const int ph = RAG ? phase_of(h + row * g.xs + g.xo) : 0;
  const int nvec = (g.C + ph + V - 1) / V;
  const int c0 = first * V - ph, cstep = W * V;  // first channel of item 0, distance of the items
  const int64_t xstep = step * g.xs, ystep = step * g.ys;
  const T* hp = h + row * g.xs + g.xo;
  const T* yp = gy + row * g.ys + g.yo;
  const T* rp = GRES ? gres + row * g.xs + g.xo : nullptr;
  T* op = gx + (gx ? row * g.xs + g.xo : 0);
  const float* sp = rstd + row;
  // rows of this thread, and of the block's first, which all of its threads walk over
  const int mine = row < g.rows ? (int)((g.rows - row + step - 1) / step) : 0;
  const int64_t left = g.rows - (int64_t)blockIdx.x * rpb;
  const int all = left > 0 ? (int)((left + step - 1) / step) : 0;
  dependents_may_start();

  bool on[NI];
  f32x2 gm[NI][P], acc[NI][P];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    on[i] = first + i * W < nvec;
#pragma unroll
    for (int e = 0; e < P; ++e) {
      gm[i][e] = both(1.f);
      acc[i][e] = 0ull;
    }
    if (gamma && on[i])
      pairs_of<T, V>(load_ends<T, V, RAG>(gamma, c0 + i * cstep, g.C), gm[i]);
  }

  auto fetch = [&](int it, uint32_t to) {  // the row that the pointers are at
    if (it < mine) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (!on[i]) continue;
        const int c = c0 + i * cstep;
        if (RAG && (c < 0 || c + V > g.C) && !inner_row(row + it * step, g.rows)) {
          write16(to + i * kLine, load_part<T, V>(hp, c, g.C));
          write16(to + (NI + i) * kLine, load_part<T, V>(yp, c, g.C));
          if (GRES) write16(to + (2 * NI + i) * kLine, load_part<T, V>(rp, c, g.C));
        } else {
          copy16(to + i * kLine, hp + c);
          copy16(to + (NI + i) * kLine, yp + c);
          if (GRES) copy16(to + (2 * NI + i) * kLine, rp + c);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    hp += xstep;
    yp += ystep;
    if (GRES) rp += xstep;
  };
  uint32_t from = slots, to = slots;
  float next_r = mine > 0 ? __ldg(sp) : 0.f;
#pragma unroll
  for (int k = 0; k < S - 1; ++k) {
    fetch(k, to);
    to += kStage;
  }
  for (int it = 0; it < all; ++it) {
    const bool live = it < mine;
    const float r = live ? next_r : 0.f;
    sp += step;
    if (it + 1 < mine) next_r = __ldg(sp);
    fetch(it + S - 1, to);
    to = to == slots + (S - 1) * kStage ? slots : to + kStage;
    asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
    R gr[NI];
    f32x2 s2 = 0ull, xh[NI][P], t[NI][P];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (!live || !on[i]) continue;
      const int c = c0 + i * cstep;
      R u = read16(from + i * kLine), w = read16(from + (NI + i) * kLine);
      if (GRES) gr[i] = read16(from + (2 * NI + i) * kLine);  // outside the row it is not used
      if (RAG && (c < 0 || c + V > g.C)) {
        clear_part<T, V>(u, c, g.C);
        clear_part<T, V>(w, c, g.C);
      }
      pairs_of<T, V>(u, xh[i]);
      pairs_of<T, V>(w, t[i]);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        xh[i][e] = mul_f32x2(xh[i][e], both(r));
        acc[i][e] = fma2(t[i][e], xh[i][e], acc[i][e]);
        t[i][e] = mul_f32x2(t[i][e], gm[i][e]);
        s2 = fma2(t[i][e], xh[i][e], s2);
      }
    }
    from = from == slots + (S - 1) * kStage ? slots : from + kStage;
    if (GRES || gx) {
      // the mean of t * (h r), negated
      const float c1 = -__fmul_rn(row_sum<NT>(sum2(s2), g.tpr, part[it & 1]), g.inv_c);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (!live || !on[i]) continue;
        f32x2 q[P];
        if (GRES) pairs_of<T, V>(gr[i], q);
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const f32x2 d = fma2(xh[i][e], both(c1), t[i][e]);
          q[e] = GRES ? fma2(d, both(r), q[e]) : mul_f32x2(d, both(r));
        }
        store_vec<T, V, RAG>(op, c0 + i * cstep, g.C, vec_of<T, V>(q));
      }
      op += xstep;
    }
  }
  if (!shares) return;
  // the block's rows in order, one line of shared memory each, then one line of the workspace
  __syncthreads();  // the lines take the slots' place
  float* lines = reinterpret_cast<float*>(dyn);  // [rpb][C]
  float* line = shares + (int64_t)blockIdx.x * g.C;
  float* to_line = rpb > 1 ? lines + grp * g.C : line;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int c = c0 + i * cstep + e;
      float lo, hi;
      unpack_f32x2(acc[i][e / 2], lo, hi);
      if (c >= 0 && c < g.C) to_line[c] = e & 1 ? hi : lo;
    }
  }
  if (rpb == 1) return;
  __syncthreads();
  for (int c = tid; c < g.C; c += NT) {
    float u = 0.f;
#pragma unroll 8
    for (int k = 0; k < rpb; ++k) u += lines[k * g.C + c];
    line[c] = u;
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
        // t * (h r), as in the rows that registers hold: t * h can leave fp32 where this does not
        if (c < g.C) s[k] = fmaf(gamma ? ld(yp + c) * ld(gamma + c) : ld(yp + c), __fmul_rn(ld(hp + c), r), s[k]);
      }
    }
    const float c1 = __fmul_rn(row_sum<kWideNT>((s[0] + s[1]) + (s[2] + s[3]), kWideNT, part), g.inv_c);
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

// ggamma[c] = the shares' sum, in a fixed order: 8 columns and 128 row lanes a
// block, each lane every 128th share; then four lanes of a warp, then the warps.
constexpr int kJoinCols = 8, kJoinLanes = 128;
template <typename T>
__global__ void __launch_bounds__(kJoinCols * kJoinLanes)
join_kernel(int C, int n, const float* __restrict__ shares, T* __restrict__ ggamma) {
  __shared__ float sm[kJoinLanes / 4][kJoinCols + 1];
  const int k = threadIdx.x % kJoinCols, l = threadIdx.x / kJoinCols, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * kJoinCols + k;
  wait_for_previous();
  float a = 0.f;
  if (c < C) {
#pragma unroll 8
    for (int b = l; b < n; b += kJoinLanes) a += shares[(int64_t)b * C + c];
  }
  a += __shfl_xor_sync(0xffffffffu, a, 8);
  a += __shfl_xor_sync(0xffffffffu, a, 16);
  if (lane < kJoinCols) sm[warp][lane] = a;
  __syncthreads();
  if (warp >= kJoinCols) return;
  a = sm[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if (lane == 0 && blockIdx.x * kJoinCols + warp < C) ggamma[blockIdx.x * kJoinCols + warp] = from_f<T>(a);
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
  int64_t n = 152 * (l.nt == 512 ? 1 : l.ni > 1 ? 2 : 3);
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

template <typename T, int V, int NI, int NT, bool RAG>
cudaError_t launch_nt(const BGeom& f, int64_t blocks, const T* h, const T* gy, const T* gamma, const float* rstd,
                      const T* gres, T* gx, float* ws, cudaStream_t s) {
  // the slots, then in their place a line of sums for each of the block's rows
  const size_t slots = (size_t)stages_of(NI) * 3 * NI * NT * 16, lines = ws && NT > f.tpr ? (size_t)(NT / f.tpr) * f.C * 4 : 0;
  const size_t smem = slots > lines ? slots : lines;
  auto kern = gres && gx ? bwd_kernel<T, V, NI, NT, RAG, true> : bwd_kernel<T, V, NI, NT, RAG, false>;
  if (smem > 46 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  kern<<<(unsigned)blocks, NT, smem, s>>>(f, h, gy, gamma, rstd, gres, gx, ws);
  return cudaGetLastError();
}
template <typename T, int V, int NI, bool RAG>
cudaError_t launch(const BGeom& f, const Lay& l, int64_t blocks, const T* h, const T* gy, const T* gamma,
                   const float* rstd, const T* gres, T* gx, float* ws, cudaStream_t s) {
  if constexpr (NI == 1) {
    return launch_nt<T, V, NI, 256, RAG>(f, blocks, h, gy, gamma, rstd, gres, gx, ws, s);
  } else {
    if constexpr (NI == 2)
      if (l.nt == 256) return launch_nt<T, V, NI, 256, RAG>(f, blocks, h, gy, gamma, rstd, gres, gx, ws, s);
    return launch_nt<T, V, NI, 512, RAG>(f, blocks, h, gy, gamma, rstd, gres, gx, ws, s);
  }
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
