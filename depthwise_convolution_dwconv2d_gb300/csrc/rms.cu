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
// shuffles of the lanes that hold a block (rows on 16 bytes). Arithmetic is on pairs of channels.
// Rows of more channels than 1024 threads hold are read twice, in spans.
//
// Rows that begin off 16 bytes (odd channels) are read in the vectors that lie
// on 16 bytes (rms.cuh): threads step over rows that begin alike. Only tensors
// that do not begin alike are read element by element.
//
// Bound by memory: 4 to 6 operations per element against 2 to 7 bytes. 16384 x
// 4096 bf16 with residual to h and e4m3 codes 78.9 us in a graph (6.0 TB/s, 0.90
// of a copy's rate), to h and y 84.7 (6.3 TB/s); one row 2.4 us.
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

template <int Q, int P>  // codes of P pairs (4 or 2)
__device__ __forceinline__ void store_codes(uint8_t* q, const f32x2* f, float inv) {
  if constexpr (P == 4)
    *reinterpret_cast<uint2*>(q) = make_uint2(encode4<Q>(f[0], f[1], inv), encode4<Q>(f[2], f[3], inv));
  else
    *reinterpret_cast<uint32_t*>(q) = encode4<Q>(f[0], f[1], inv);
}
__device__ __forceinline__ uint32_t max_bits(uint32_t m, f32x2 v) {
  return max(m, max((uint32_t)v & 0x7fffffffu, (uint32_t)(v >> 32) & 0x7fffffffu));
}

// The codes' blocks k0 and k1 of the V channels from c on, of which the first
// `cut` are k0's (k1 = k0 and cut = V where there is one block).
struct Span { int k0, k1, cut; };
template <int V>
__device__ __forceinline__ Span span_of(int c, int C, int shift) {
  Span s;
  s.k0 = max(c, 0) >> shift;
  s.k1 = min(c + V, C) - 1 >> shift;
  s.cut = s.k1 > s.k0 ? (s.k1 << shift) - c : V;
  return s;
}

// ---- rows that 256 or 512 threads hold ---------------------------------------------

constexpr int kNT = 256;
__device__ uint4 kNone[1];  // read in place of what does not exist
// Blocks step over the rows; the next row's vectors are on their way while one
// is worked on. RAG: rows begin anywhere and the step is a multiple of 8 of
// them; the maxima of the codes' blocks meet in shared memory (the largest of
// bit patterns: in any order the same). Brought together by shuffles first they
// took longer (6000 x 2131 fp16 with residual to codes 76 us against 63.5; from
// a copy of the row, a warp each, 41 against 39 at 13470 x 723, and no row of
// more than 1016 channels). 512 threads: rows of 1025 to 2048
// vectors, of which a block of 1024 threads to a row by itself, without the
// next row on its way, took 34.5 us for 1432 x 4736 fp32 with residual, to codes.
template <typename T, int V, int NI, int Q, bool RAG, int NT = kNT>
__global__ void __launch_bounds__(NT, NT > kNT ? 1 : NI == 1 ? 4 : NI == 2 ? 3 : 2)
fwd_rows_kernel(FGeom g, const T* x, const T* res, const T* __restrict__ gamma, T* h, T* y, float* rstd, Act8 t) {
  typedef typename Raw<T, V>::type R;
  constexpr int P = V / 2;
  constexpr bool kSplit = RAG && Q != kSrcFull;  // a block of codes begins anywhere in a vector
  __shared__ float part[2][NT / 32];
  __shared__ uint32_t maxima[2][kSplit ? NT * NI * V / 32 + NT / 4 : 1];  // of the codes' blocks, for each row in turn
  const int tid = threadIdx.x;
  const int in_row = tid & (g.tpr - 1);
  const int W = NI > 1 || g.tpr >= 32 ? 32 : g.tpr;  // rows of fewer than 32 lanes have one vector a lane
  const int st = NI > 1 ? g.tpr : 32;  // from item to item, in vectors: all warps have as many; in channels:
  const int cst = st * V;
  const int rpb = NT >> g.log_tpr;
  const int64_t step = (int64_t)gridDim.x * rpb;
  int64_t row = (int64_t)blockIdx.x * rpb + (tid >> g.log_tpr);
  const int ph = RAG ? phase_of(x + row * g.xs + g.xo) : 0;
  const int nvec = (g.C + ph + V - 1) / V;
  const int c0 = in_row * V - ph;  // first channel of item 0
  const int64_t xstep = step * g.xs, ystep = step * g.ys;
  const T* xp = x + row * g.xs + g.xo;
  const T* rp = res + (res ? row * g.xs + g.xo : 0);
  T* hp = h + (h ? row * g.xs + g.xo : 0);
  T* yp = y + (y ? row * g.ys + g.yo : 0);
  f32x2 gm[NI][P];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
#pragma unroll
    for (int e = 0; e < P; ++e) gm[i][e] = both(1.f);
    if (gamma && in_row + i * st < nvec)
      pairs_of<T, V>(load_ends<T, V, RAG>(gamma, c0 + i * cst, g.C), gm[i]);
  }
  R nx[NI], nr[NI];
  auto over = [&](int i) { return RAG && (c0 + i * cst < 0 || c0 + i * cst + V > g.C); };  // the row's ends
  // The row that the pointers are at. Nothing here uses what is read, and no
  // read hangs on a condition (one that does not exist reads zeros instead):
  // both made the reads wait for one another (3073 x 2130 fp32: 63.6 us, 24.0
  // without). Vectors over the tensor's ends are read where they are used.
  auto fetch = [&](int64_t at) {
    const bool inner = inner_row(at, g.rows);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const bool no = at >= g.rows || in_row + i * st >= nvec || (RAG && !inner && over(i));
      nx[i] = *(no ? (const R*)kNone : reinterpret_cast<const R*>(xp + c0 + i * cst));
      if (res) nr[i] = *(no ? (const R*)kNone : reinterpret_cast<const R*>(rp + c0 + i * cst));
    }
  };
  const int line = (tid >> g.log_tpr) * t.nblk;  // of the maxima
  if constexpr (kSplit) {
    for (int k = tid; k < rpb * t.nblk; k += NT) maxima[0][k] = maxima[1][k] = 0;
    __syncthreads();
  }
  // where x's rows are as far apart as the codes', their vectors are whole ones too
  const bool whole = kSplit && (reinterpret_cast<uintptr_t>(t.codes) + row * g.C - ph) % V == 0;
  int flip = 0;
  fetch(row);
  for (int64_t base = (int64_t)blockIdx.x * rpb; base < g.rows; base += step, row += step, flip ^= 1) {
    const bool live = row < g.rows;
    R hv[NI];
    f32x2 s2 = 0ull;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (!live || in_row + i * st >= nvec) continue;
      f32x2 a[P];
      const bool apart = over(i) && !inner_row(row, g.rows);
      if (apart) hv[i] = load_part<T, V>(xp, c0 + i * cst, g.C);
      else hv[i] = nx[i];
      if (res) {
        R rv;
        if (apart) rv = load_part<T, V>(rp, c0 + i * cst, g.C);
        else rv = nr[i];
        f32x2 b[P];
        pairs_of<T, V>(hv[i], a);
        pairs_of<T, V>(rv, b);
#pragma unroll
        for (int e = 0; e < P; ++e) a[e] = add_f32x2(a[e], b[e]);
        hv[i] = vec_of<T, V>(a);
      }
      if (over(i)) clear_part<T, V>(hv[i], c0 + i * cst, g.C);
      pairs_of<T, V>(hv[i], a);
#pragma unroll
      for (int e = 0; e < P; ++e) s2 = fma2(a[e], a[e], s2);
    }
    xp += xstep;
    rp += xstep;
    // the next row is read before this one's h is written: x or the residual may be h's memory, row by row
    fetch(row + step);
    if (h) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (live && in_row + i * st < nvec) store_vec<T, V, RAG>(hp, c0 + i * cst, g.C, hv[i]);
      hp += xstep;
    }
    const float ss = row_sum<NT>(sum2(s2), g.tpr, part[flip]);
    const float r = __frsqrt_rn(fmaf(ss, g.inv_c, g.eps));
    if (live && in_row == 0 && rstd) rstd[row] = r;
    uint32_t* mx = maxima[flip] + (kSplit ? line : 0);
    if constexpr (kSplit) {
      if (g.tpr <= 32) __syncwarp();
      for (int k = in_row; k < t.nblk; k += g.tpr) maxima[flip ^ 1][line + k] = 0;  // the next row's
    }
    {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const bool on = live && in_row + i * st < nvec;
        f32x2 f[P];
#pragma unroll
        for (int e = 0; e < P; ++e) f[e] = 0ull;
        if (on) {
          pairs_of<T, V>(hv[i], f);
#pragma unroll
          for (int e = 0; e < P; ++e) f[e] = mul_f32x2(mul_f32x2(f[e], both(r)), gm[i][e]);
          if (y) store_vec<T, V, RAG>(yp, c0 + i * cst, g.C, vec_of<T, V>(f));
        }
        if constexpr (kSplit) {
          const Span b = span_of<V>(c0 + i * cst, g.C, t.shift);
          uint32_t m = 0;
          if (b.k1 == b.k0) {
#pragma unroll
            for (int e = 0; e < P; ++e) m = max_bits(m, f[e]);
          } else {
            uint32_t m1 = 0;
#pragma unroll
            for (int e = 0; e < P; ++e) {
              const uint32_t lo = (uint32_t)f[e] & 0x7fffffffu, hi = (uint32_t)(f[e] >> 32) & 0x7fffffffu;
              m = max(m, max(2 * e < b.cut ? lo : 0, 2 * e + 1 < b.cut ? hi : 0));
              m1 = max(m1, max(2 * e < b.cut ? 0 : lo, 2 * e + 1 < b.cut ? 0 : hi));
            }
            if (on) atomicMax(mx + b.k1, m1);
          }
          if (on) atomicMax(mx + b.k0, m);
        } else if constexpr (Q != kSrcFull) {
          uint32_t m = 0;
#pragma unroll
          for (int e = 0; e < P; ++e) m = max_bits(m, f[e]);
          const int block = 1 << t.shift;
          for (int o = min(block / V, W) >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          if (on) {
            const int c = c0 + i * cst;
            float inv;
            const float s = scale_of<Q>(m, &inv);
            store_codes<Q, P>(t.codes + row * g.C + c, f, inv);
            if ((c & (block - 1)) == 0) t.scales[row * t.nblk + (c >> t.shift)] = s;
          }
        }
      }
      yp += ystep;
    }
    if constexpr (kSplit) {
      if (g.tpr <= 32) __syncwarp();
      else __syncthreads();
      uint8_t* q = t.codes + row * g.C;
      float* sc = t.scales + row * t.nblk;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (!live || in_row + i * st >= nvec) continue;
        const int c = c0 + i * cst;
        const Span b = span_of<V>(c, g.C, t.shift);
        float inv0, inv1;
        const float s0 = scale_of<Q>(mx[b.k0], &inv0);
        inv1 = inv0;
        if (b.k1 != b.k0) sc[b.k1] = scale_of<Q>(mx[b.k1], &inv1);
        if (c <= b.k0 << t.shift) sc[b.k0] = s0;
        f32x2 f[P];
        pairs_of<T, V>(hv[i], f);
#pragma unroll
        for (int e = 0; e < P; ++e) {
          f[e] = mul_f32x2(mul_f32x2(f[e], both(r)), gm[i][e]);
          f[e] = mul_f32x2(f[e], pack_f32x2(2 * e < b.cut ? inv0 : inv1, 2 * e + 1 < b.cut ? inv0 : inv1));
        }
        uint32_t w[2] = {encode4<Q>(f[0], f[1], 1.f), 0};
        if constexpr (V == 8) w[1] = encode4<Q>(f[2], f[3], 1.f);
        uint8_t* at = q + c;
        if (c >= 0 && c + V <= g.C && whole) {
          if constexpr (V == 8) *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
          else *reinterpret_cast<uint32_t*>(at) = w[0];
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e)
            if (c + e >= 0 && c + e < g.C) at[e] = (uint8_t)(w[e / 4] >> (8 * (e & 3)));
        }
      }
    }
  }
}

// ---- wider rows, on 16 bytes ---------------------------------------------------------

// A block to a row: few rows, of 257 to 512 vectors by 512 threads and to 2048
// by 1024, where latency counts; and rows of over 2048 vectors, read twice (the
// second time mostly from L2: 2000 x 30000 bf16 with residual 91 us, 72 the floor).
template <typename T, int V, int NI, int Q, int NT>
__global__ void __launch_bounds__(NT)
fwd_wide_kernel(FGeom g, const T* x, const T* res, const T* __restrict__ gamma, T* h, T* y, float* rstd, Act8 t) {
  typedef typename Raw<T, V>::type R;
  constexpr int P = V / 2;
  __shared__ float part[NT / 32];
  const int tid = threadIdx.x;
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
    // the second read of a row takes h where it was stored: x or the residual may be the same memory
    const bool stored = again && h;
    R rv[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int v = seg * span + first + i * W;
      if (live && v < g.nvec) {
        hv[i] = *reinterpret_cast<const R*>((stored ? hr : xr) + (int64_t)v * V);
        if (res && !stored) rv[i] = *reinterpret_cast<const R*>(rr + (int64_t)v * V);
      }
    }
    if (res && !stored) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        f32x2 a[P], b[P];
        pairs_of<T, V>(hv[i], a);
        pairs_of<T, V>(rv[i], b);
#pragma unroll
        for (int e = 0; e < P; ++e) a[e] = add_f32x2(a[e], b[e]);
        hv[i] = vec_of<T, V>(a);
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
    f32x2 s2 = 0ull;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (!live || seg * span + first + i * W >= g.nvec) continue;
      f32x2 a[P];
      pairs_of<T, V>(hv[i], a);
#pragma unroll
      for (int e = 0; e < P; ++e) s2 = fma2(a[e], a[e], s2);
    }
    ss += sum2(s2);
  }
  ss = row_sum<NT>(ss, g.tpr, part);
  const float r = __frsqrt_rn(fmaf(ss, g.inv_c, g.eps));
  if (live && in_row == 0 && rstd) rstd[row] = r;

  T* yr = y + (y ? row * g.ys + g.yo : 0);
  for (int seg = 0; seg < g.segs; ++seg) {
    if (g.segs > 1) {
      load_gamma(seg);
      load_h(seg, true);
    }
    const f32x2 r2 = both(r);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int v = seg * span + first + i * W;
      const bool on = live && v < g.nvec;
      f32x2 f[P];
#pragma unroll
      for (int e = 0; e < P; ++e) f[e] = 0ull;
      if (on) {
        pairs_of<T, V>(hv[i], f);
#pragma unroll
        for (int e = 0; e < P; ++e) f[e] = mul_f32x2(f[e], r2);
        if (gamma) {
          f32x2 gm[P];
          pairs_of<T, V>(gv[i], gm);
#pragma unroll
          for (int e = 0; e < P; ++e) f[e] = mul_f32x2(f[e], gm[e]);
        }
        if (y) *reinterpret_cast<R*>(yr + (int64_t)v * V) = vec_of<T, V>(f);
      }
      if constexpr (Q != kSrcFull) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < P; ++e) m = max_bits(m, f[e]);
        const int block = 1 << t.shift;
        for (int o = min(block / V, W) >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (on) {
          const int c = v * V;
          float inv;
          const float s = scale_of<Q>(m, &inv);
          store_codes<Q, P>(t.codes + row * g.C + c, f, inv);
          if ((c & (block - 1)) == 0) t.scales[row * t.nblk + (c >> t.shift)] = s;
        }
      }
    }
  }
}

// ---- element by element --------------------------------------------------------------

template <typename T, int Q, int NT>
__global__ void __launch_bounds__(NT)
fwd_elem_kernel(FGeom g, const T* x, const T* res, const T* __restrict__ gamma, T* h, T* y,
           float* rstd, Act8 t) {
  constexpr int V = 1, NI = 8;
  typedef T R;
  __shared__ float part[NT / 32];
  const int tid = threadIdx.x;
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
  ss = row_sum<NT>(ss, g.tpr, part);
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
        *q = encode1<Q>(f[i][0], inv);
        if ((c & (block - 1)) == 0) t.scales[row * t.nblk + (c >> t.shift)] = s;
      }
    }
  }
}

// ---- host -------------------------------------------------------------------------------

void spread(Lay* l, int64_t nvec, int most) {
  const int64_t need = (nvec + l->ni - 1) / l->ni;
  l->tpr = pow2_at_least(need);
  if (l->tpr < 4) l->tpr = 4;
  if (l->tpr > most) l->tpr = most;
  l->segs = (int)((need + l->tpr - 1) / l->tpr);
}

// Vectors per thread: one while all rows together are less than a wave of
// threads (latency counts), else two, or four where 256 or 512 threads then hold a row.
Lay lay(const Rms& g, int V) {
  Lay l{};
  l.v = V;
  const int64_t nvec = g.C / V;
  const bool wave = g.rows * nvec > 152 * 2048;
  l.ni = !wave && nvec <= 1024 ? 1 : nvec <= 64 ? 1 : nvec <= 512 ? 2 : nvec <= 1024 || (wave && nvec <= 2048) ? 4 : 2;
  spread(&l, nvec, 1024);
  l.nt = l.tpr > kNT ? l.tpr : kNT;
  return l;
}
Lay lay_elem(const Rms& g) {
  Lay l{};
  l.v = 1;
  l.ni = 8;
  spread(&l, g.C, 1024);
  l.nt = l.tpr > 256 ? l.tpr : 256;
  return l;
}
// segs > 1: not one for the ragged form.
Lay lay_ragged(const Rms& g, int V) {
  Lay l{};
  l.v = V;
  const int64_t nvec = (g.C + 2 * V - 2) / V;
  l.ni = 1;
  const int most = g.rows * nvec > 152 * 2048 ? 64 : kNT;  // as above: latency counts
  while (l.ni < 4 && l.ni * most < nvec) l.ni *= 2;
  spread(&l, nvec, 2 * kNT);
  if (l.ni > 1 && l.tpr < 32) l.tpr = 32;
  l.nt = l.tpr > kNT ? l.tpr : kNT;
  return l;
}

struct Args {
  const void *x, *res, *gamma;
  void *h, *y;
  float* rstd;
  Act8 t;
};

FGeom geom(const Rms& g, const Lay& l) {
  FGeom f{};
  f.rows = g.rows;
  f.xs = g.xs; f.xo = g.xo; f.ys = g.ys; f.yo = g.yo;
  f.C = g.C;
  f.nvec = g.C / l.v;
  f.tpr = l.tpr;
  while ((1 << f.log_tpr) < l.tpr) ++f.log_tpr;
  f.segs = l.segs;
  f.eps = g.eps;
  f.inv_c = 1.f / (float)g.C;
  return f;
}

template <typename T, int Q, typename KernelT>
cudaError_t launch(KernelT kern, const Rms& g, const Lay& l, const Args& a, cudaStream_t s) {
  FGeom f = geom(g, l);
  const int64_t rpb = l.nt / l.tpr, most = (int64_t(1) << 30) * rpb;
  for (int64_t r = 0; r < g.rows; r += most) {  // grids of at most 2^30 blocks
    f.rows = g.rows - r < most ? g.rows - r : most;
    Act8 u = a.t;
    if (Q != kSrcFull) {
      u.codes += r * g.C;
      u.scales += r * u.nblk;
    }
    const int64_t ox = r * g.xs, oy = r * g.ys;
    kern<<<(unsigned)((f.rows + rpb - 1) / rpb), l.nt, 0, s>>>(
        f, (const T*)a.x + ox, a.res ? (const T*)a.res + ox : nullptr, (const T*)a.gamma, a.h ? (T*)a.h + ox : nullptr,
        a.y ? (T*)a.y + oy : nullptr, a.rstd ? a.rstd + r : nullptr, u);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T, int Q, bool RAG>
cudaError_t run_rows(const Rms& g, const Lay& l, const Args& a, cudaStream_t s) {
  constexpr int V = Vec<T>::n;
  const int64_t rpb = l.nt / l.tpr, all = (g.rows + rpb - 1) / rpb;
  const int64_t held = 152 * (l.nt > kNT ? 1 : l.ni == 1 ? 4 : l.ni == 2 ? 3 : 2);  // by the kernels' registers: one wave
  int64_t blocks = all < held ? all : held;
  while (blocks * rpb % 8) ++blocks;
  const FGeom f = geom(g, l);
  const auto kern = l.nt > kNT  ? fwd_rows_kernel<T, V, 4, Q, RAG, 2 * kNT>
                    : l.ni == 1 ? fwd_rows_kernel<T, V, 1, Q, RAG>
                    : l.ni == 2 ? fwd_rows_kernel<T, V, 2, Q, RAG>
                                : fwd_rows_kernel<T, V, 4, Q, RAG>;
  kern<<<(unsigned)blocks, l.nt, 0, s>>>(f, (const T*)a.x, (const T*)a.res, (const T*)a.gamma, (T*)a.h, (T*)a.y, a.rstd, a.t);
  return cudaGetLastError();
}

template <typename T, int Q>
cudaError_t run(const Rms& g, const Args& a, cudaStream_t s) {
  constexpr int V = Vec<T>::n;
  if (rows_on16(g, V) && on16(a.x) && on16(a.res) && on16(a.gamma) && on16(a.h) && on16(a.y) &&
      (Q == kSrcFull || reinterpret_cast<uintptr_t>(a.t.codes) % V == 0)) {
    const Lay l = lay(g, V);
    if (l.nt == kNT || l.ni == 4) return run_rows<T, Q, false>(g, l, a, s);
    if (l.nt == 512) return launch<T, Q>(fwd_wide_kernel<T, V, 1, Q, 512>, g, l, a, s);
    return launch<T, Q>(l.ni == 1 ? fwd_wide_kernel<T, V, 1, Q, 1024> : fwd_wide_kernel<T, V, 2, Q, 1024>, g, l, a, s);
  }
  const Lay l = lay_ragged(g, V);
  if (l.segs == 1 && alike(a.x, a.res) && alike(a.x, a.h) && alike(a.x, a.y) && (!a.y || rows_alike(g, V)))
    return run_rows<T, Q, true>(g, l, a, s);
  const Lay e = lay_elem(g);
  if (e.nt == 256) return launch<T, Q>(fwd_elem_kernel<T, Q, 256>, g, e, a, s);
  if (e.nt == 512) return launch<T, Q>(fwd_elem_kernel<T, Q, 512>, g, e, a, s);
  return launch<T, Q>(fwd_elem_kernel<T, Q, 1024>, g, e, a, s);
}

}  // namespace

bool fwd_in_row(const Rms& g) {
  const int V = g.dtype == DWCONV_F32 ? 4 : 8;
  if (rows_on16(g, V)) return lay(g, V).segs == 1;
  return (lay_ragged(g, V).segs == 1 && rows_alike(g, V)) || lay_elem(g).segs == 1;
}

cudaError_t fwd(const Rms& g, const void* x, const void* residual, const void* gamma, void* h, void* y, float* rstd,
                const Act8& t, cudaStream_t s) {
  if (g.rows == 0) return cudaSuccess;
  const Args a{x, residual, gamma, h, y, rstd, t};
  cudaError_t e = cudaErrorInvalidValue;
  if (!t.codes) {
    DWCONV_DISPATCH_DTYPE(g.dtype, T, e = run<T, kSrcFull>(g, a, s));
  } else if (t.src == kSrcI8) {
    DWCONV_DISPATCH_DTYPE(g.dtype, T, e = run<T, kSrcI8>(g, a, s));
  } else {
    DWCONV_DISPATCH_DTYPE(g.dtype, T, e = run<T, kSrcE4M3>(g, a, s));
  }
  return e;
}

}  // namespace rms
}  // namespace dwconv
