// 1x1 layers over 8-bit floats on the tensor cores (formula: pointwise8.cu).
//
// A block of 128 channels is 128 bytes of a row: one row of the 128-byte
// swizzle, four tcgen05.mma of K = 32. Its sum is left in tensor memory by
// itself, read back and added, times its two scales, to fp32 sums in
// registers: the scales are any fp32 values, which no MMA applies. Two
// accumulators take turns, so that a block's MMAs run while the one before is
// read back.
//
// Tile kernel (many pixels): a tile is 128 pixels (M) x 128 or 256 outputs
// (N). Roles: a producer lane (tensor-map copies), an MMA warp, and a
// warpgroup per 128 outputs that reads back and adds: a thread has one pixel
// and 128 outputs, hence one scale of x and one of w per block. Persistent.
//
// Row kernel (few pixels, where the weights are all there is to read): the
// roles of the operands are swapped, 128 outputs (M) x 16 to 128 pixels (N),
// and a cluster of up to 8 thread blocks shares the channels' blocks of a
// tile, so that all SMs read weights. Their sums are joined through the
// cluster's shared memory in a fixed order.
//
// Every wait is bounded; a wait that gives up raises the block's abort flag
// and every role then runs through its loops without waiting, waits (bounded)
// for its own copies and MMAs in flight, frees the tensor memory and returns.
#include <atomic>

#include <cooperative_groups.h>

#include "norm.cuh"
#include "pointwise8.h"
#include "tc.cuh"
#include "vec.cuh"

namespace dwconv {
namespace pw8 {
namespace {

namespace cg = cooperative_groups;

constexpr unsigned kSleepNs = 32;

// Instruction descriptor of kind::f8f6f4, e4m3 x e4m3 with fp32 D, both operands K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

__device__ __forceinline__ void mma_f8(uint32_t dtmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(dtmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A block of 128 channels: four steps of 32, 32 bytes (2 descriptor units) apart. One thread.
__device__ __forceinline__ void mma_block(uint32_t dtmem, const void* a, const void* b, uint32_t idesc) {
  const uint64_t ad = tc::desc_sw128(tma::smem_u32(a)), bd = tc::desc_sw128(tma::smem_u32(b));
#pragma unroll
  for (int k = 0; k < 4; ++k) mma_f8(dtmem, ad + 2 * k, bd + 2 * k, idesc, k > 0 ? 1u : 0u);
}

// 32 or 16 consecutive fp32 columns of this warp's 32 lanes, one lane per thread, as pairs; not waited for
__device__ __forceinline__ void ld_pairs32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void ld_pairs16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// Waits for this thread's loads; naming the registers keeps their uses behind the wait.
__device__ __forceinline__ void ld_wait32(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               ::"memory");
}
__device__ __forceinline__ void ld_wait16(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               ::"memory");
}
__device__ __forceinline__ f32x2 pair_at(const uint32_t* r, int i) { return ((f32x2)r[2 * i + 1] << 32) | r[2 * i]; }

struct Ring {
  int s = 0;
  uint32_t ph = 0;
  bool wrapped = false;
  __device__ __forceinline__ void next(int stages) {
    if (++s == stages) { s = 0; ph ^= 1; wrapped = true; }
  }
};

__device__ __forceinline__ unsigned char* align1024(unsigned char* p) { return p + ((1024 - (tma::smem_u32(p) & 1023)) & 1023); }

// V values of y's row from column c on: bias, activation, one rounding
template <typename T, int V>
__device__ __forceinline__ void finish(const Pw& g, const T* bias, int c, float* v) {
  if (bias) {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] += ld(bias + (c + e < g.cout ? c + e : c));
  }
  norm::act_v<V>(g.act, v);
}

// ---- tile kernel --------------------------------------------------------------

constexpr int kM = 128;

template <int BN>
struct Tile {
  static constexpr int kEpi = BN;               // threads that read back
  static constexpr int kThreads = kEpi + 64;    // and a producer and an MMA warp
  static constexpr int kStages = 4;
  static constexpr int kA = kM * kBlock, kB = BN * kBlock, kStage = kA + kB;
  static constexpr int kCols = 2 * BN;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage;
  static constexpr int kPerSm = BN == 128 ? 1 : 1;
};

struct TGeom {
  Pw p;
  int tiles;       // below 2^31
  FastDiv d_nt;    // tiles across the outputs
  int vec_out;
};

template <typename T, int BN>
__global__ void __launch_bounds__(Tile<BN>::kThreads, Tile<BN>::kPerSm)
tile_kernel(TGeom g, const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
            unsigned int* timeouts, const float* __restrict__ sx, const float* __restrict__ sw,
            const T* __restrict__ bias, T* __restrict__ y) {
  typedef Tile<BN> K;
  extern __shared__ unsigned char smdyn[];
  __shared__ __align__(8) uint64_t full[K::kStages], empty[K::kStages], accfull[2], accfree[2], done;
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_s;
  unsigned char* sm = align1024(smdyn);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kProducer = K::kEpi / 32, kMma = kProducer + 1;
  if (tid == 0) {
    for (int s = 0; s < K::kStages; ++s) {
      tma::mbar_init(&full[s], 1);
      tma::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      tma::mbar_init(&accfull[s], 1);
      tma::mbar_init(&accfree[s], K::kEpi / 32);
    }
    tma::mbar_init(&done, 1);
    tma::fence_init();
    abort_s = 0;
  }
  if (warp == kMma) tc::alloc(&tmem_base_s, K::kCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_base_s;
  volatile int* abortp = &abort_s;
  const int nkb = g.p.nkb;

  if (warp == kProducer) {
    if (lane == 0) {
      Ring r;
      uint32_t issued = 0;
      for (int t = blockIdx.x; t < g.tiles && !*abortp; t += gridDim.x) {
        uint32_t mt;
        const int nt = (int)g.d_nt.divmod((uint32_t)t, mt);
        for (int kb = 0; kb < nkb && !*abortp; ++kb, r.next(K::kStages)) {
          if (r.wrapped && !tc::wait(&empty[r.s], r.ph ^ 1, timeouts, abortp)) { *abortp = 1; break; }
          unsigned char* st = sm + (size_t)r.s * K::kStage;
          tma::mbar_expect_tx(&full[r.s], K::kStage);
          tma::load_3d(st, &xmap, kb * kBlock, (int)mt * kM, 0, &full[r.s]);
          tma::load_3d(st + K::kA, &wmap, kb * kBlock, nt * BN, 0, &full[r.s]);
          ++issued;
        }
      }
      // every issued copy lands before the block leaves
      const uint32_t first = issued > (uint32_t)K::kStages ? issued - K::kStages : 0;
      for (uint32_t k = first; k < issued; ++k) tc::wait(&full[k % K::kStages], (k / K::kStages) & 1, nullptr, nullptr);
    }
    __syncwarp();
  } else if (warp == kMma) {
    constexpr uint32_t idesc = idesc_e4m3(kM, BN);
    Ring r;
    uint32_t it = 0;
    for (int t = blockIdx.x; t < g.tiles; t += gridDim.x) {
      for (int kb = 0; kb < nkb; ++kb, ++it, r.next(K::kStages)) {
        const int ab = it & 1;
        const bool ok = !*abortp && (it < 2 || tc::wait(&accfree[ab], ((it >> 1) - 1) & 1, timeouts, abortp)) &&
                        tc::wait(&full[r.s], r.ph, timeouts, abortp);
        if (!__all_sync(0xffffffffu, ok)) { *abortp = 1; continue; }
        tc::fence_after();
        const unsigned char* st = sm + (size_t)r.s * K::kStage;
        if (tc::elect_one()) {
          mma_block(tmem + ab * BN, st, st + K::kA, idesc);
          tc::commit(&empty[r.s]);
          tc::commit(&accfull[ab]);
        }
        __syncwarp();
      }
    }
    if (tc::elect_one()) tc::commit(&done);
    __syncwarp();
    tc::wait(&done, 0, nullptr, nullptr);
    __syncwarp();
  } else {
    const int col0 = (warp >> 2) * 128;  // this warpgroup's outputs of the tile
    const uint32_t tlane = tmem + ((uint32_t)((warp & 3) * 32) << 16) + col0;
    uint32_t it = 0;
    for (int t = blockIdx.x; t < g.tiles; t += gridDim.x) {
      uint32_t mt;
      const int nt = (int)g.d_nt.divmod((uint32_t)t, mt);
      const int64_t p = (int64_t)mt * kM + (warp & 3) * 32 + lane;
      const int o0 = nt * BN + col0;
      const bool valid = p < g.p.rows && o0 < g.p.cout;
      const float* sxp = sx + (valid ? p * nkb : 0);
      const float* swp = sw + (int64_t)(valid ? o0 / kBlock : 0) * nkb;
      float sxn = __ldg(sxp), swn = __ldg(swp);
      f32x2 acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0ull;
      for (int kb = 0; kb < nkb; ++kb, ++it) {
        const int ab = it & 1;
        const float sc = __fmul_rn(sxn, swn);
        if (kb + 1 < nkb) {
          sxn = __ldg(sxp + kb + 1);
          swn = __ldg(swp + kb + 1);
        }
        const f32x2 s2 = pack_f32x2(sc, sc);
        bool ok = !*abortp && tc::wait(&accfull[ab], (it >> 1) & 1, timeouts, abortp);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) *abortp = 1;
        tc::fence_after();
        if (ok) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t d[32];
            ld_pairs32(tlane + ab * BN + 32 * q, d);
            ld_wait32(d);
#pragma unroll
            for (int i = 0; i < 16; ++i) fma_f32x2(acc[16 * q + i], pair_at(d, i), s2);
          }
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::arrive(&accfree[ab]);
      }
      if (!valid || *abortp) continue;
      T* yp = y + p * g.p.ys + g.p.yo;
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int c = o0 + 8 * q;
        if (c >= g.p.cout) break;
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) unpack_f32x2(acc[4 * q + i], v[2 * i], v[2 * i + 1]);
        finish<T, 8>(g.p, bias, c, v);
        if (g.vec_out && c + 8 <= g.p.cout) {
          uint4* dst = reinterpret_cast<uint4*>(yp + c);
          dst[0] = pack16<T>(v);
          if constexpr (sizeof(T) == 4) dst[1] = pack16<T>(v + 4);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + e < g.p.cout) yp[c + e] = from_f<T>(v[e]);
        }
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMma) tc::dealloc(tmem, K::kCols);
}

// ---- row kernel ------------------------------------------------------------------

template <int NP>
struct Row {
  static constexpr int kThreads = 128 + 64;
  static constexpr int kA = 128 * kBlock, kB = NP * kBlock, kStage = kA + kB;
  static constexpr int kStages = NP <= 32 ? 5 : NP == 64 ? 4 : 3;  // two blocks fit an SM
  static constexpr int kCols = 2 * NP < 32 ? 32 : 2 * NP;
  static constexpr int kTab = 32 * 1024;  // the block's scales, at most
  static constexpr size_t kJoin = (size_t)NP * 128 * 4;
  static_assert(kJoin <= (size_t)kStages * kStage, "the joined sums take the stages' place");
};

struct RGeom {
  Pw p;
  int split;  // thread blocks of a cluster, which share the channels' blocks
};

template <typename T, int NP>
__global__ void __launch_bounds__(Row<NP>::kThreads)
row_kernel(RGeom g, const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
           unsigned int* timeouts, const float* __restrict__ sx, const float* __restrict__ sw,
           const T* __restrict__ bias, T* __restrict__ y) {
  typedef Row<NP> K;
  extern __shared__ unsigned char smdyn[];
  __shared__ __align__(8) uint64_t full[K::kStages], empty[K::kStages], accfull[2], accfree[2], done;
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_s;
  unsigned char* sm = align1024(smdyn);
  float* tab = reinterpret_cast<float*>(sm + (size_t)K::kStages * K::kStage);  // [block of channels][pixel]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kProducer = 4, kMma = 5;
  const int rank = blockIdx.x % g.split, o0 = blockIdx.x / g.split * 128;
  const int64_t p0 = (int64_t)blockIdx.y * NP;
  const int nkb = g.p.nkb;
  const int kb0 = rank * nkb / g.split, kb1 = (rank + 1) * nkb / g.split;
  if (tid == 0) {
    for (int s = 0; s < K::kStages; ++s) {
      tma::mbar_init(&full[s], 1);
      tma::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      tma::mbar_init(&accfull[s], 1);
      tma::mbar_init(&accfree[s], 4);
    }
    tma::mbar_init(&done, 1);
    tma::fence_init();
    abort_s = 0;
  }
  if (warp == kMma) tc::alloc(&tmem_base_s, K::kCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_base_s;
  volatile int* abortp = &abort_s;
  f32x2 acc[NP / 2];

  if (warp == kProducer) {
    if (lane == 0) {
      Ring r;
      uint32_t issued = 0;
      for (int kb = kb0; kb < kb1 && !*abortp; ++kb, r.next(K::kStages)) {
        if (r.wrapped && !tc::wait(&empty[r.s], r.ph ^ 1, timeouts, abortp)) { *abortp = 1; break; }
        unsigned char* st = sm + (size_t)r.s * K::kStage;
        tma::mbar_expect_tx(&full[r.s], K::kStage);
        tma::load_3d(st, &wmap, kb * kBlock, o0, 0, &full[r.s]);
        tma::load_3d(st + K::kA, &xmap, kb * kBlock, (int)p0, 0, &full[r.s]);
        ++issued;
      }
      const uint32_t first = issued > (uint32_t)K::kStages ? issued - K::kStages : 0;
      for (uint32_t k = first; k < issued; ++k) tc::wait(&full[k % K::kStages], (k / K::kStages) & 1, nullptr, nullptr);
    }
    __syncwarp();
  } else if (warp == kMma) {
    constexpr uint32_t idesc = idesc_e4m3(128, NP);
    Ring r;
    for (int it = 0; it < kb1 - kb0; ++it, r.next(K::kStages)) {
      const int ab = it & 1;
      const bool ok = !*abortp && (it < 2 || tc::wait(&accfree[ab], ((it >> 1) - 1) & 1, timeouts, abortp)) &&
                      tc::wait(&full[r.s], r.ph, timeouts, abortp);
      if (!__all_sync(0xffffffffu, ok)) { *abortp = 1; continue; }
      tc::fence_after();
      const unsigned char* st = sm + (size_t)r.s * K::kStage;
      if (tc::elect_one()) {
        mma_block(tmem + ab * NP, st, st + K::kA, idesc);
        tc::commit(&empty[r.s]);
        tc::commit(&accfull[ab]);
      }
      __syncwarp();
    }
    if (tc::elect_one()) tc::commit(&done);
    __syncwarp();
    tc::wait(&done, 0, nullptr, nullptr);
    __syncwarp();
  } else {
    // the products of the scales, while the first copies are on their way
    for (int i = tid; i < (kb1 - kb0) * NP; i += 128) {
      const int kb = kb0 + i / NP;
      const int64_t p = p0 + i % NP;
      tab[i] = p < g.p.rows ? __fmul_rn(__ldg(sx + p * nkb + kb), __ldg(sw + (int64_t)(o0 / kBlock) * nkb + kb)) : 0.f;
    }
    asm volatile("bar.sync 1, 128;\n" ::: "memory");
#pragma unroll
    for (int i = 0; i < NP / 2; ++i) acc[i] = 0ull;
    const uint32_t tlane = tmem + ((uint32_t)(warp * 32) << 16);
    for (int it = 0; it < kb1 - kb0; ++it) {
      const int ab = it & 1;
      bool ok = !*abortp && tc::wait(&accfull[ab], (it >> 1) & 1, timeouts, abortp);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) *abortp = 1;
      tc::fence_after();
      if (ok) {
        const float* tp = tab + it * NP;
#pragma unroll
        for (int q = 0; q < NP / 16; ++q) {
          uint32_t d[16];
          ld_pairs16(tlane + ab * NP + 16 * q, d);
          ld_wait16(d);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(tp + 16 * q + 4 * i);
            fma_f32x2(acc[8 * q + 2 * i], pair_at(d, 2 * i), s.x);
            fma_f32x2(acc[8 * q + 2 * i + 1], pair_at(d, 2 * i + 1), s.y);
          }
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::arrive(&accfree[ab]);
    }
  }
  tc::fence_before();
  __syncthreads();  // all copies have landed and all MMAs are done: the stages are free
  tc::fence_after();
  if (warp == kMma) tc::dealloc(tmem, K::kCols);

  // Sums of all blocks of the cluster, in order of the channels; each block finishes a share of the pixels.
  float* mine = reinterpret_cast<float*>(sm);  // [pixel][output]
  const int n = (int)(g.p.rows - p0 < NP ? g.p.rows - p0 : NP);
  if (warp < 4) {
#pragma unroll
    for (int i = 0; i < NP / 2; ++i) {
      float a, b;
      unpack_f32x2(acc[i], a, b);
      if (2 * i < n) mine[(2 * i) * 128 + tid] = a;
      if (2 * i + 1 < n) mine[(2 * i + 1) * 128 + tid] = b;
    }
  }
  cg::cluster_group cl = cg::this_cluster();
  cl.sync();
  if (warp < 4 && o0 + tid < g.p.cout) {
    const int lo = rank * n / g.split, hi = (rank + 1) * n / g.split;
    for (int p = lo; p < hi; ++p) {
      float v = 0.f;
      for (int k = 0; k < g.split; ++k) v += *cl.map_shared_rank(mine + p * 128 + tid, k);
      finish<T, 1>(g.p, bias, o0 + tid, &v);
      y[(p0 + p) * g.p.ys + g.p.yo + o0 + tid] = from_f<T>(v);
    }
  }
  cl.sync();  // no block leaves while others read its sums
}

// ---- host ---------------------------------------------------------------------------

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// Rows of `cols` bytes, ld bytes apart; boxes of 128 bytes x box_rows with the
// 128-byte swizzle, zeros outside. (A third dimension of one plane: the copies are tma::load_3d.)
bool encode_bytes(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint64_t ld, uint32_t box_rows) {
  EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cols, rows, 1};
  const cuuint64_t strides[2] = {ld, ld * rows};
  const cuuint32_t box[3] = {kBlock, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A kernel's shared-memory limit, raised once per device
template <typename KernelT>
cudaError_t allow_smem(KernelT kern, size_t smem, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && dev < 64) done.fetch_or(uint64_t(1) << dev, std::memory_order_release);
  return e;
}

int64_t tiles_of(const Pw& g, int bn) { return ((g.rows + kM - 1) / kM) * ((g.cout + bn - 1) / bn); }

template <typename T, int BN>
cudaError_t launch_tile(const Pw& g, int64_t ldx, const uint8_t* x, const float* sx, const uint8_t* w, const float* sw,
                        const T* bias, T* y, cudaStream_t s) {
  typedef Tile<BN> K;
  alignas(64) CUtensorMap xmap{}, wmap{};
  if (!encode_bytes(&xmap, x, (uint64_t)(ldx == g.pitch ? g.pitch : g.cin), (uint64_t)g.rows, (uint64_t)ldx, kM) ||
      !encode_bytes(&wmap, w, (uint64_t)g.pitch, (uint64_t)g.cout, (uint64_t)g.pitch, BN))
    return cudaErrorNotSupported;
  unsigned int* to = tma::timeout_counter();
  if (!to) return cudaErrorNotSupported;
  static std::atomic<uint64_t> ready{0};
  auto kern = tile_kernel<T, BN>;
  cudaError_t e = allow_smem(kern, K::kSmem, ready);
  if (e != cudaSuccess) return e;
  TGeom t{};
  t.p = g;
  t.tiles = (int)tiles_of(g, BN);
  t.d_nt = FastDiv((uint32_t)((g.cout + BN - 1) / BN));
  const int es = (int)sizeof(T);
  t.vec_out = g.ys * es % 16 == 0 && g.yo * es % 16 == 0 && reinterpret_cast<uintptr_t>(y) % 16 == 0;
  const int most = 152 * K::kPerSm;
  kern<<<t.tiles < most ? t.tiles : most, K::kThreads, K::kSmem, s>>>(t, xmap, wmap, to, sx, sw, bias, y);
  return cudaGetLastError();
}

// Thread blocks that share a tile's channels: as many as give every SM two,
// each at least two blocks of channels.
int split_of(const Pw& g, int np) {
  const int64_t tiles = (int64_t)((g.cout + 127) / 128) * ((g.rows + np - 1) / np);
  int n = 1;
  while (n < 8 && tiles * n * 2 <= 152 * 2 && g.nkb >= 4 * n) n *= 2;
  return n;
}

template <typename T, int NP>
cudaError_t launch_row(const Pw& g, int64_t ldx, const uint8_t* x, const float* sx, const uint8_t* w, const float* sw,
                       const T* bias, T* y, cudaStream_t s) {
  typedef Row<NP> K;
  alignas(64) CUtensorMap xmap{}, wmap{};
  if (!encode_bytes(&xmap, x, (uint64_t)(ldx == g.pitch ? g.pitch : g.cin), (uint64_t)g.rows, (uint64_t)ldx, NP) ||
      !encode_bytes(&wmap, w, (uint64_t)g.pitch, (uint64_t)g.cout, (uint64_t)g.pitch, 128))
    return cudaErrorNotSupported;
  unsigned int* to = tma::timeout_counter();
  if (!to) return cudaErrorNotSupported;
  static std::atomic<uint64_t> ready{0};
  auto kern = row_kernel<T, NP>;
  constexpr size_t most = 1024 + (size_t)K::kStages * K::kStage + K::kTab;
  cudaError_t e = allow_smem(kern, most, ready);
  if (e != cudaSuccess) return e;
  RGeom r{};
  r.p = g;
  r.split = split_of(g, NP);
  const int held = (g.nkb + r.split - 1) / r.split;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)r.split;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((g.cout + 127) / 128 * r.split), (unsigned)((g.rows + NP - 1) / NP));
  cfg.blockDim = dim3(K::kThreads);
  cfg.dynamicSmemBytes = 1024 + (size_t)K::kStages * K::kStage + (size_t)held * NP * 4;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, r, (const CUtensorMap)xmap, (const CUtensorMap)wmap, to, sx, sw, bias, y);
  return e != cudaSuccess ? e : cudaGetLastError();
}

int row_pixels(const Pw& g) { return g.rows <= 16 ? 16 : g.rows <= 32 ? 32 : g.rows <= 64 ? 64 : 128; }

template <typename T>
cudaError_t run_t(const Pw& g, int64_t ldx, const uint8_t* x, const float* sx, const uint8_t* w, const float* sw,
                  const T* bias, T* y, cudaStream_t s) {
  if (plan(g) == Plan::Row) {
    switch (row_pixels(g)) {
      case 16: return launch_row<T, 16>(g, ldx, x, sx, w, sw, bias, y, s);
      case 32: return launch_row<T, 32>(g, ldx, x, sx, w, sw, bias, y, s);
      case 64: return launch_row<T, 64>(g, ldx, x, sx, w, sw, bias, y, s);
      default: return launch_row<T, 128>(g, ldx, x, sx, w, sw, bias, y, s);
    }
  }
  if (tiles_of(g, 128) >= (int64_t(1) << 31)) return cudaErrorNotSupported;
  if (tiles_of(g, 256) >= 152) return launch_tile<T, 256>(g, ldx, x, sx, w, sw, bias, y, s);
  return launch_tile<T, 128>(g, ldx, x, sx, w, sw, bias, y, s);
}

}  // namespace

Plan plan(const Pw& g) {
  if (g.rows > 128) return Plan::Tile;
  const int np = row_pixels(g), split = split_of(g, np);
  return (int64_t)((g.nkb + split - 1) / split) * np * 4 <= 32 * 1024 ? Plan::Row : Plan::Tile;
}

cudaError_t run_tc(const Pw& g, int64_t ldx, const uint8_t* x, const float* sx, const uint8_t* w, const float* sw,
                   const void* bias, void* y, cudaStream_t s) {
  if (g.rows >= (int64_t(1) << 31) - 256) return cudaErrorNotSupported;  // coordinates of a copy are 32 bits
  cudaError_t e = cudaErrorInvalidValue;
  DWCONV_DISPATCH_DTYPE(g.dtype, T, e = run_t<T>(g, ldx, x, sx, w, sw, (const T*)bias, (T*)y, s));
  return e;
}

}  // namespace pw8
}  // namespace dwconv
