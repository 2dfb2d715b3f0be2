// 1x1 layers over 8-bit floats on the tensor cores (formula: pointwise8.cu).
//
// A block of 128 channels is 128 bytes of a row: one row of the 128-byte
// swizzle, four tcgen05.mma of K = 32. Its sum is left in tensor memory by
// itself, read back and added, times its two scales, to fp32 sums in
// registers: the scales are any fp32 values, which no MMA applies. Two
// accumulators take turns, so that a block's MMAs run while the one before is
// read back.
//
// Tile kernels (many pixels): 128 pixels (M) x 128 outputs (N) by a thread
// block, or 256 x 256 by a pair of them. Roles: two producer lanes (tensor-map
// copies; one lane's follow one another, 491 cycles for 128 rows of 128 bytes,
// so one of them would hold 32 KB a stage to 983), an MMA warp, and warps that
// read back and add: a thread has one pixel and 64 or 128 outputs, hence one
// scale of x and one of w per block. Persistent.
//
// Row kernel (few pixels, where the weights are all there is to read): the
// roles of the operands are swapped, 128 outputs (M) x 16 to 64 pixels (N),
// and a cluster of up to 8 thread blocks shares the channels' blocks of a
// tile, so that all SMs read weights. Their sums are joined through the
// cluster's shared memory in a fixed order.
//
// Every wait is bounded; a wait that gives up raises the block's abort flag
// and every role then runs through its loops without waiting, waits (bounded)
// for its own copies and MMAs in flight, frees the tensor memory and returns.
#include <atomic>

#include <cooperative_groups.h>

#include "dependent.cuh"
#include "norm.cuh"
#include "pointwise8.h"
#include "tc.cuh"
#include "vec.cuh"

namespace dwconv {
namespace pw8 {
namespace {

namespace cg = cooperative_groups;

// Instruction descriptor of kind::f8f6f4, e4m3 x e4m3 with fp32 D, both operands K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

template <int CTAS>
__device__ __forceinline__ void mma_f8(uint32_t dtmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  if constexpr (CTAS == 1) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(dtmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(dtmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

// A block of 128 channels: four steps of 32, 32 bytes (2 descriptor units) apart. One thread.
template <int CTAS>
__device__ __forceinline__ void mma_block(uint32_t dtmem, const void* a, const void* b, uint32_t idesc) {
  const uint64_t ad = tc::desc_sw128(tma::smem_u32(a)), bd = tc::desc_sw128(tma::smem_u32(b));
#pragma unroll
  for (int k = 0; k < 4; ++k) mma_f8<CTAS>(dtmem, ad + 2 * k, bd + 2 * k, idesc, k > 0 ? 1u : 0u);
}

// 16 consecutive fp32 columns of this warp's 32 lanes, one lane per thread, as pairs; not waited for
__device__ __forceinline__ void ld_pairs16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// Waits for this thread's loads; naming the registers keeps their uses behind the wait.
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

// Before a block leaves, every copy that a producer issued has landed (those of
// a stage that both have issued to), and so has every arrival that frees one of
// its stages: those of the last STAGES nobody else waits for, and in a pair
// they come from the other block. full: null where the copies count elsewhere.
// After a give-up the arrivals may never come and are not waited for.
template <int STAGES>
__device__ __forceinline__ void drain(uint64_t* full, uint64_t* empty, uint32_t issued, volatile int* abortp) {
  const uint32_t first = issued > (uint32_t)STAGES ? issued - STAGES : 0;
  for (uint32_t k = first; k < issued; ++k) {
    if (full) tc::wait(&full[k % STAGES], (k / STAGES) & 1, nullptr, nullptr);
    tc::wait(&empty[k % STAGES], (k / STAGES) & 1, nullptr, abortp);
  }
}

// One of two MMA warps: the blocks of channels which, which + 2, ... of `total`
// of this thread block's. A warp by itself takes 900 cycles from one to the
// next (two barriers of 200 each, issue and commits 350), longer than the MMAs.
// issue(accumulator, stage) runs in one lane and commits.
template <int STAGES, int ACC, typename Issue>
__device__ __forceinline__ void mma_loop(int which, uint32_t total, uint64_t* full, uint64_t* accfree, unsigned int* timeouts,
                                         volatile int* abortp, Issue issue) {
  Ring r;
  if (which) r.next(STAGES);
  for (uint32_t it = which; it < total; it += 2) {
    const int ab = it % ACC;
    const bool ok = tc::wait(&full[r.s], r.ph, timeouts, abortp) &&
                    (it < ACC || tc::wait(&accfree[ab], (it / ACC - 1) & 1, timeouts, abortp));
    if (__all_sync(0xffffffffu, ok)) {
      tc::fence_after();
      if (tc::elect_one()) issue(ab, r.s);
      __syncwarp();
    } else {
      *abortp = 1;
    }
    r.next(STAGES);
    r.next(STAGES);
  }
}

__device__ __forceinline__ unsigned char* align1024(unsigned char* p) { return p + ((1024 - (tma::smem_u32(p) & 1023)) & 1023); }

// ---- tile kernels -------------------------------------------------------------

constexpr int kM = 128;  // pixels of a thread block

struct TGeom {
  Pw p;
  int tiles;       // below 2^31
  FastDiv d_nt;    // tiles across the outputs
  int vec_out;
};

// acc += s * (NC columns of this warp's lanes), 16 at a time. freed() runs once all have been read.
template <int NC, typename F>
__device__ __forceinline__ void add_block(uint32_t taddr, f32x2 s2, f32x2* acc, F freed) {
#pragma unroll
  for (int q = 0; q < NC / 16; ++q) {
    uint32_t d[16];
    ld_pairs16(taddr + 16 * q, d);
    ld_wait16(d);
    if (q + 1 == NC / 16) freed();
#pragma unroll
    for (int i = 0; i < 8; ++i) fma_f32x2(acc[8 * q + i], pair_at(d, i), s2);
  }
}

// 32 bytes of a row, on 32 bytes
__device__ __forceinline__ void store32(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
               "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// 16 columns of this warp's 32 lanes back to tensor memory
__device__ __forceinline__ void st_pairs16(uint32_t taddr, const f32x2* v) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r[2 * i] = (uint32_t)v[i];
    r[2 * i + 1] = (uint32_t)(v[i] >> 32);
  }
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// The sums of a warp's 32 pixels x NC outputs (a thread has a pixel) to y:
// bias, activation, one rounding; a thread stores 32 bytes of its row at a
// time. Rows off 32 bytes go through 2 KB of shared memory instead, so that
// neighbouring lanes store neighbouring elements. The sums are read from the
// accumulator that they came from last (taddr, which is not free yet), times
// s2: those of more than one block of channels were put back there, because
// registers cannot be indexed: the code for all columns in a row took longer
// to fetch than the sums to compute, and its registers cost the loop over the
// channels its own.
constexpr int kSt = 16;                        // columns at a time
constexpr int warp_floats(int nc) { return 32 * kSt + nc; }  // staging and bias of a warp
template <typename T, int NC>
__device__ __forceinline__ void store_tile(const TGeom& g, T* y, int p0, int o0, uint32_t taddr, f32x2 s2, float* st) {
  const int lane = threadIdx.x & 31;
  const int rows = min((int)g.p.rows - p0, 32);  // at most 0: nothing to store
  const int cols = rows > 0 ? g.p.cout - o0 : 0;
  const float* bias = st + 32 * kSt;
  T* yr = y + (int64_t)(p0 + lane) * g.p.ys + g.p.yo + o0;
#pragma unroll 1
  for (int c0 = 0; c0 < NC && c0 < cols; c0 += 32) {
    uint32_t d[32];
    ld_pairs16(taddr + c0, d);
    ld_pairs16(taddr + c0 + 16, d + 16);
    ld_wait16(d);
    ld_wait16(d + 16);
    f32x2 u[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(bias + c0 + 4 * i);
      u[2 * i] = norm::fma2(pair_at(d, 2 * i), s2, b.x);
      u[2 * i + 1] = norm::fma2(pair_at(d, 2 * i + 1), s2, b.y);
    }
    norm::act_p<16>(g.p.act, u);
    if (g.vec_out && c0 + 32 <= cols) {
      if (lane < rows) {
        float v[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) unpack_f32x2(u[i], v[2 * i], v[2 * i + 1]);
        constexpr int VEC = Vec<T>::n;
#pragma unroll
        for (int i = 0; i < 32; i += 2 * VEC) store32(yr + c0 + i, pack16<T>(v + i), pack16<T>(v + i + VEC));
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // a pixel's four 16-byte groups, each moved by its pixel: lanes do not meet in a bank
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<ulonglong2*>(st + lane * kSt + ((j ^ (lane >> 1)) & 3) * 4) =
              make_ulonglong2(u[8 * h + 2 * j], u[8 * h + 2 * j + 1]);
        __syncwarp();
        const int k = lane & 15, c = c0 + kSt * h + k;
        if (c < cols) {
          T* yp = y + (int64_t)(p0 + (lane >> 4)) * g.p.ys + g.p.yo + o0 + c;
#pragma unroll 8
          for (int i = 0; i < 16; ++i) {
            const int r = 2 * i + (lane >> 4);
            if (r < rows) yp[2 * i * g.p.ys] = from_f<T>(st[r * kSt + (((k >> 2) ^ (r >> 1)) & 3) * 4 + (k & 3)]);
          }
        }
        __syncwarp();
      }
    }
  }
}

// What a warp that reads back needs of a tile before its first block of
// channels: fetched while the tile before it is stored.
template <typename T, int NC>
struct Ahead {
  float sx, sw, bias[NC / 32];
  __device__ __forceinline__ void fetch(const Pw& p, const float* sx_, const float* sw_, const T* b, int p0, int o0) {
    const int lane = threadIdx.x & 31;
    sx = __ldg(sx_ + (p0 + lane < (int)p.rows ? (int64_t)(p0 + lane) * p.nkb : 0));
    sw = __ldg(sw_ + (o0 < p.cout ? o0 / kBlock : 0) * p.nkb);
#pragma unroll
    for (int k = 0; k < NC / 32; ++k) bias[k] = b && o0 + 32 * k + lane < p.cout ? ld(b + o0 + 32 * k + lane) : 0.f;
  }
  __device__ __forceinline__ void put_bias(float* st) const {
    __syncwarp();
#pragma unroll
    for (int k = 0; k < NC / 32; ++k) st[32 * kSt + 32 * k + (threadIdx.x & 31)] = bias[k];
    __syncwarp();
  }
};

// A warp that reads back, over its tiles: tile t's first pixel and output from
// at(t, p0, o0), whose accumulators are n columns apart from tlane on.
template <typename T, int NC, int ACC, typename At, typename Free>
__device__ __forceinline__ void read_back(const TGeom& g, const float* sx, const float* sw, const T* bias, T* y, int first,
                                          int step, uint32_t tlane, int n, float* st, uint64_t* accfull,
                                          unsigned int* timeouts, volatile int* abortp, At at, Free free_acc) {
  const int lane = threadIdx.x & 31, nkb = g.p.nkb;
  uint32_t it = 0;
  int p0, o0;
  Ahead<T, NC> a;
  if (first < g.tiles) {
    at(first, p0, o0);
    a.fetch(g.p, sx, sw, bias, p0, o0);
  }
  for (int t = first; t < g.tiles; t += step) {
    a.put_bias(st);
    const float* sxp = sx + (p0 + lane < (int)g.p.rows ? (int64_t)(p0 + lane) * nkb : 0);
    const float* swp = sw + (o0 < g.p.cout ? o0 / kBlock : 0) * nkb;
    f32x2 acc[NC / 2];
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) acc[i] = 0ull;
    f32x2 s2 = 0ull;
    for (int kb = 0; kb < nkb; ++kb, ++it) {
      const float sc = __fmul_rn(a.sx, a.sw);
      s2 = pack_f32x2(sc, sc);
      if (kb + 1 < nkb) {
        a.sx = __ldg(sxp + kb + 1);
        a.sw = __ldg(swp + kb + 1);
      }
      bool ok = tc::wait(&accfull[it % ACC], (it / ACC) & 1, timeouts, abortp);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) *abortp = 1;
      tc::fence_after();
      auto freed = [&] {
        if (kb + 1 < nkb) free_acc(it % ACC);  // the last one is still needed
      };
      if (ok && nkb > 1) add_block<NC>(tlane + (it % ACC) * n, s2, acc, freed);
      else freed();
    }
    const int last = (it - 1) % ACC;
    const int tp0 = p0, to0 = o0;
    if (nkb > 1) {
#pragma unroll
      for (int q = 0; q < NC / 16; ++q) st_pairs16(tlane + last * n + 16 * q, acc + 8 * q);
      asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
      s2 = pack_f32x2(1.f, 1.f);
    }
    if (t + step < g.tiles) {
      at(t + step, p0, o0);
      a.fetch(g.p, sx, sw, bias, p0, o0);
    }
    if (!*abortp) store_tile<T, NC>(g, y, tp0, to0, tlane + last * n, s2, st);
    free_acc(last);
  }
}

// One thread block, 128 pixels x 128 outputs, for calls of few tiles: four
// accumulators take turns here, so that neither the MMAs nor the warps that
// read back wait for the other's hand-over.
struct Tile {
  static constexpr int kN = 128, kNC = 64;        // outputs of a tile, of a warp that reads back
  static constexpr int kAcc = 4;                   // accumulators (a power of two)
  static constexpr int kEpi = 4 * kN / kNC;       // warps that read back
  static constexpr int kThreads = 32 * kEpi + 128;  // and two producers and two MMA warps
  static constexpr int kStages = 6;
  static constexpr int kA = kM * kBlock, kB = kN * kBlock, kStage = kA + kB;
  static constexpr int kCols = kAcc * kN;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + kEpi * warp_floats(kNC) * 4;
};

template <typename T>
__global__ void __launch_bounds__(Tile::kThreads, 1)
tile_kernel(TGeom g, const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
            unsigned int* timeouts, const float* __restrict__ sx, const float* __restrict__ sw,
            const T* __restrict__ bias, T* __restrict__ y) {
  typedef Tile K;
  extern __shared__ unsigned char smdyn[];
  __shared__ __align__(8) uint64_t full[K::kStages], empty[K::kStages], accfull[K::kAcc], accfree[K::kAcc], done;
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_s;
  unsigned char* sm = align1024(smdyn);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kProducer = K::kEpi, kMma = kProducer + 2;
  if (tid == 0) {
    for (int s = 0; s < K::kStages; ++s) {
      tma::mbar_init(&full[s], 1);
      tma::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < K::kAcc; ++s) {
      tma::mbar_init(&accfull[s], 1);
      tma::mbar_init(&accfree[s], K::kEpi);
    }
    tma::mbar_init(&done, 2);  // both MMA warps
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

  if (warp == kProducer || warp == kProducer + 1) {
    if (lane == 0) {
      const bool first_one = warp == kProducer;  // x's copies, and the bytes of both; the other one w's
      if (first_one) wait_for_previous();  // the aligned copy of x
      Ring r;
      uint32_t issued = 0;
      for (int t = blockIdx.x; t < g.tiles && !*abortp; t += gridDim.x) {
        uint32_t mt;
        const int nt = (int)g.d_nt.divmod((uint32_t)t, mt);
        for (int kb = 0; kb < nkb && !*abortp; ++kb, r.next(K::kStages)) {
          if (r.wrapped && !tc::wait(&empty[r.s], r.ph ^ 1, timeouts, abortp)) { *abortp = 1; break; }
          unsigned char* st = sm + (size_t)r.s * K::kStage;
          if (first_one) {
            tma::mbar_expect_tx(&full[r.s], K::kStage);
            tma::load_3d(st, &xmap, kb * kBlock, (int)mt * kM, 0, &full[r.s]);
          } else {
            tma::load_3d(st + K::kA, &wmap, kb * kBlock, nt * K::kN, 0, &full[r.s]);
          }
          ++issued;
        }
      }
      drain<K::kStages>(full, empty, issued, abortp);
    }
    __syncwarp();
  } else if (warp >= kMma) {
    constexpr uint32_t idesc = idesc_e4m3(kM, K::kN);
    const uint32_t mine = (int)blockIdx.x < g.tiles ? (g.tiles - 1 - blockIdx.x) / gridDim.x + 1 : 0;
    mma_loop<K::kStages, K::kAcc>(warp - kMma, mine * nkb, full, accfree, timeouts, abortp, [&](int ab, int stage) {
      const unsigned char* st = sm + (size_t)stage * K::kStage;
      mma_block<1>(tmem + ab * K::kN, st, st + K::kA, idesc);
      tc::commit(&empty[stage]);
      tc::commit(&accfull[ab]);
    });
    if (tc::elect_one()) tc::commit(&done);
    __syncwarp();
    tc::wait(&done, 0, nullptr, nullptr);
    __syncwarp();
  } else {
    const int col0 = (warp >> 2) * K::kNC;  // this warp's outputs of the tile; its pixels are 32 (warp % 4) and on
    const uint32_t tlane = tmem + ((uint32_t)((warp & 3) * 32) << 16) + col0;
    float* st = reinterpret_cast<float*>(sm + (size_t)K::kStages * K::kStage) + warp * warp_floats(K::kNC);
    read_back<T, K::kNC, K::kAcc>(
        g, sx, sw, bias, y, blockIdx.x, gridDim.x, tlane, K::kN, st, accfull, timeouts, abortp,
        [&](int t, int& p0, int& o0) {
          uint32_t mt;
          o0 = (int)g.d_nt.divmod((uint32_t)t, mt) * K::kN + col0;
          p0 = (int)mt * kM + (warp & 3) * 32;
        },
        [&](int ab) {
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::arrive(&accfree[ab]);
        });
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == kMma) tc::dealloc(tmem, K::kCols);
}

// A pair of thread blocks on two SMs, 256 pixels x 256 outputs: each holds
// its 128 pixels and half of the weights, and one MMA reads both. That is 32 KB
// per block of channels and SM where a block by itself reads 48 for 128 x 256.
struct Pair {
  static constexpr int kN = 256, kNC = 128;
  static constexpr int kAcc = 2;
  static constexpr int kEpi = 4 * kN / kNC;        // warps that read back
  static constexpr int kThreads = 32 * kEpi + 128;  // and a warpgroup of two producers and two MMA warps
  static constexpr int kStages = 6;
  static constexpr int kA = kM * kBlock, kB = kN / 2 * kBlock, kStage = kA + kB;
  static constexpr int kCols = kAcc * kN;
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + kEpi * warp_floats(kNC) * 4;
};

// A copy that counts on the barrier of the pair's first block
__device__ __forceinline__ void load_pair(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(tma::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(0), "r"(tma::smem_u32(bar) & 0xFEFFFFFFu)
      : "memory");
}
// Arrive on bar in both blocks of the pair once every tcgen05 operation so far is done
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(
                   tma::smem_u32(bar)),
               "h"((uint16_t)3)
               : "memory");
}
// Arrive on bar of the pair's first block
__device__ __forceinline__ void arrive_first(uint64_t* bar) {
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, 0;\n"
      " mbarrier.arrive.shared::cluster.b64 _, [a];\n}\n" ::"r"(tma::smem_u32(bar))
      : "memory");
}

template <typename T>
__global__ void __launch_bounds__(Pair::kThreads, 1) __cluster_dims__(2, 1, 1)
pair_kernel(TGeom g, const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
            unsigned int* timeouts, const float* __restrict__ sx, const float* __restrict__ sw,
            const T* __restrict__ bias, T* __restrict__ y) {
  typedef Pair K;
  extern __shared__ unsigned char smdyn[];
  __shared__ __align__(8) uint64_t full[K::kStages], empty[K::kStages], accfull[K::kAcc], accfree[K::kAcc], done;
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_s;
  unsigned char* sm = align1024(smdyn);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int kProducer = K::kEpi, kMma = kProducer + 2;
  const int rank = blockIdx.x & 1;  // in the pair; block 0 issues the MMAs and has the barriers they wait for
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (tid == 0) {
    for (int s = 0; s < K::kStages; ++s) {
      tma::mbar_init(&full[s], 1);
      tma::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < K::kAcc; ++s) {
      tma::mbar_init(&accfull[s], 1);
      tma::mbar_init(&accfree[s], 2 * K::kEpi);  // the warps of both blocks that read back
    }
    tma::mbar_init(&done, 2);  // both MMA warps
    tma::fence_init();
    abort_s = 0;
  }
  if (warp == kMma) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(tma::smem_u32(&tmem_base_s)),
                 "r"(K::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
  }
  tc::fence_before();
  cg::this_cluster().sync();
  tc::fence_after();
  const uint32_t tmem = tmem_base_s;
  volatile int* abortp = &abort_s;
  const int nkb = g.p.nkb;

  if (warp >= K::kEpi) {
    // of the 168 registers a thread that the block was launched with: 128 x 56 + 256 x 224 = 384 x 168
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;\n");
    if (warp == kProducer || warp == kProducer + 1) {
      if (lane == 0) {
        const bool first_one = warp == kProducer;  // x's copies, and block 0's the bytes of all; the other one w's
        if (first_one) wait_for_previous();  // the aligned copy of x
        Ring r;
        uint32_t issued = 0;
        for (int t = pair; t < g.tiles && !*abortp; t += pairs) {
          uint32_t mt;
          const int nt = (int)g.d_nt.divmod((uint32_t)t, mt);
          for (int kb = 0; kb < nkb && !*abortp; ++kb, r.next(K::kStages)) {
            if (r.wrapped && !tc::wait(&empty[r.s], r.ph ^ 1, timeouts, abortp)) { *abortp = 1; break; }
            unsigned char* st = sm + (size_t)r.s * K::kStage;
            if (first_one) {
              if (rank == 0) tma::mbar_expect_tx(&full[r.s], 2 * K::kStage);
              load_pair(st, &xmap, kb * kBlock, ((int)mt * 2 + rank) * kM, &full[r.s]);
            } else {
              load_pair(st + K::kA, &wmap, kb * kBlock, nt * K::kN + rank * (K::kN / 2), &full[r.s]);
            }
            ++issued;
          }
        }
        drain<K::kStages>(rank == 0 ? full : nullptr, empty, issued, abortp);
      }
      __syncwarp();
    } else {
      if (rank == 0) {
        constexpr uint32_t idesc = idesc_e4m3(2 * kM, K::kN);
        const uint32_t mine = pair < g.tiles ? (g.tiles - 1 - pair) / pairs + 1 : 0;
        mma_loop<K::kStages, K::kAcc>(warp - kMma, mine * nkb, full, accfree, timeouts, abortp, [&](int ab, int stage) {
          const unsigned char* st = sm + (size_t)stage * K::kStage;
          mma_block<2>(tmem + ab * K::kN, st, st + K::kA, idesc);
          commit_pair(&empty[stage]);
          commit_pair(&accfull[ab]);
        });
        if (tc::elect_one()) commit_pair(&done);
        __syncwarp();
      }
      tc::wait(&done, 0, nullptr, nullptr);  // block 1 too: its MMAs' ends arrive from block 0
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;\n");
    const int col0 = (warp >> 2) * K::kNC;  // this warp's outputs of the tile; its pixels are 32 (warp % 4) and on
    const uint32_t tlane = tmem + ((uint32_t)((warp & 3) * 32) << 16) + col0;
    float* st = reinterpret_cast<float*>(sm + (size_t)K::kStages * K::kStage) + warp * warp_floats(K::kNC);
    read_back<T, K::kNC, K::kAcc>(
        g, sx, sw, bias, y, pair, pairs, tlane, K::kN, st, accfull, timeouts, abortp,
        [&](int t, int& p0, int& o0) {
          uint32_t mt;
          o0 = (int)g.d_nt.divmod((uint32_t)t, mt) * K::kN + col0;
          p0 = ((int)mt * 2 + rank) * kM + (warp & 3) * 32;
        },
        [&](int ab) {
          tc::fence_before();
          __syncwarp();
          if (lane == 0) arrive_first(&accfree[ab]);
        });
  }
  tc::fence_before();
  // Neither block leaves while the other's MMAs, copies or arrivals may reach it.
  // This orders the threads; what they started is waited for before: copies,
  // freed stages (drain), sums (every accfull by the warps that read back) and
  // done, in both blocks.
  cg::this_cluster().sync();
  tc::fence_after();
  if (warp == kMma)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(K::kCols) : "memory");
}

// ---- row kernel ------------------------------------------------------------------

template <int NP>
struct Row {
  static constexpr int kThreads = 128 + 128;  // a warpgroup that reads back, two producers and two MMA warps
  static constexpr int kA = 128 * kBlock, kB = NP * kBlock, kStage = kA + kB;
  static constexpr int kStages = NP <= 32 ? 5 : 4;  // two blocks fit an SM
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
  constexpr int kProducer = 4, kMma = 6;
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
    tma::mbar_init(&done, 2);  // both MMA warps
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

  if (warp == kProducer || warp == kProducer + 1) {
    if (lane == 0) {
      const bool first_one = warp == kProducer;  // w's copies, and the bytes of both; the other one x's
      if (!first_one) wait_for_previous();  // the aligned copy of x
      Ring r;
      uint32_t issued = 0;
      for (int kb = kb0; kb < kb1 && !*abortp; ++kb, r.next(K::kStages)) {
        if (r.wrapped && !tc::wait(&empty[r.s], r.ph ^ 1, timeouts, abortp)) { *abortp = 1; break; }
        unsigned char* st = sm + (size_t)r.s * K::kStage;
        if (first_one) {
          tma::mbar_expect_tx(&full[r.s], K::kStage);
          tma::load_3d(st, &wmap, kb * kBlock, o0, 0, &full[r.s]);
        } else {
          tma::load_3d(st + K::kA, &xmap, kb * kBlock, (int)p0, 0, &full[r.s]);
        }
        ++issued;
      }
      drain<K::kStages>(full, empty, issued, abortp);
    }
    __syncwarp();
  } else if (warp >= kMma) {
    constexpr uint32_t idesc = idesc_e4m3(128, NP);
    mma_loop<K::kStages, 2>(warp - kMma, kb1 - kb0, full, accfree, timeouts, abortp, [&](int ab, int stage) {
      const unsigned char* st = sm + (size_t)stage * K::kStage;
      mma_block<1>(tmem + ab * NP, st, st + K::kA, idesc);
      tc::commit(&empty[stage]);
      tc::commit(&accfull[ab]);
    });
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
      bool ok = tc::wait(&accfull[ab], (it >> 1) & 1, timeouts, abortp);
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
  if (warp < 4) {
    // Sums are whole only if no block of the cluster gave up: otherwise nothing
    // is stored, as in the tile kernels. A lane looks at one block's flag; the
    // read is on its way beside those of the first sums (waited for before
    // them it took 0.25 of 6 us, 0.08 here).
    const int gave_up = lane < g.split ? *cl.map_shared_rank(&abort_s, lane) : 0;
    bool whole = false;
    const bool in = o0 + tid < g.p.cout;
    const int lo = rank * n / g.split, hi = (rank + 1) * n / g.split;
    const float b = bias && in ? ld(bias + o0 + tid) : 0.f;
    T* yp = y + p0 * g.p.ys + g.p.yo + o0 + tid;
#pragma unroll 1
    for (int p = lo; p < hi; p += 4) {  // four pixels' reads at a time
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = 0.f;
      for (int k = 0; k < g.split; ++k) {
        const float* theirs = cl.map_shared_rank(mine + tid, k);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (p + e < hi) v[e] += theirs[(p + e) * 128];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += b;
      norm::act_v<4>(g.p.act, v);
      if (p == lo) whole = __all_sync(0xffffffffu, gave_up == 0);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (whole && in && p + e < hi) yp[(p + e) * g.p.ys] = from_f<T>(v[e]);
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

int64_t tiles_of(const Pw& g, int m, int n) { return ((g.rows + m - 1) / m) * ((g.cout + n - 1) / n); }

// KERN: tile_kernel or pair_kernel, of which K is the shape
template <typename K, typename T, typename KernelT>
cudaError_t launch_tiles(KernelT kern, bool pair, std::atomic<uint64_t>& ready, const Pw& g, int64_t ldx, const uint8_t* x,
                         bool copied, const float* sx, const uint8_t* w, const float* sw, const T* bias, T* y, cudaStream_t s) {
  alignas(64) CUtensorMap xmap{}, wmap{};
  if (!encode_bytes(&xmap, x, (uint64_t)(ldx == g.pitch ? g.pitch : g.cin), (uint64_t)g.rows, (uint64_t)ldx, kM) ||
      !encode_bytes(&wmap, w, (uint64_t)g.pitch, (uint64_t)g.cout, (uint64_t)g.pitch, K::kB / kBlock))
    return cudaErrorNotSupported;
  unsigned int* to = tma::timeout_counter();
  if (!to) return cudaErrorNotSupported;
  cudaError_t e = allow_smem(kern, K::kSmem, ready);
  if (e != cudaSuccess) return e;
  TGeom t{};
  t.p = g;
  t.tiles = (int)tiles_of(g, pair ? 2 * kM : kM, K::kN);
  t.d_nt = FastDiv((uint32_t)((g.cout + K::kN - 1) / K::kN));
  const int es = (int)sizeof(T);
  t.vec_out = g.ys * es % 32 == 0 && g.yo * es % 32 == 0 && reinterpret_cast<uintptr_t>(y) % 32 == 0;
  const int most = pair ? 76 : 152;
  const int n = t.tiles < most ? t.tiles : most;
  if (copied)
    return launch_dependent(kern, dim3(pair ? 2 * n : n), dim3(K::kThreads), K::kSmem, s, t, (const CUtensorMap)xmap,
                            (const CUtensorMap)wmap, to, sx, sw, bias, y);
  kern<<<pair ? 2 * n : n, K::kThreads, K::kSmem, s>>>(t, xmap, wmap, to, sx, sw, bias, y);
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
cudaError_t launch_row(const Pw& g, int64_t ldx, const uint8_t* x, bool copied, const float* sx, const uint8_t* w, const float* sw,
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
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)r.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // dependent.cuh
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((g.cout + 127) / 128 * r.split), (unsigned)((g.rows + NP - 1) / NP));
  cfg.blockDim = dim3(K::kThreads);
  cfg.dynamicSmemBytes = 1024 + (size_t)K::kStages * K::kStage + (size_t)held * NP * 4;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = copied ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, r, (const CUtensorMap)xmap, (const CUtensorMap)wmap, to, sx, sw, bias, y);
  return e != cudaSuccess ? e : cudaGetLastError();
}

int row_pixels(const Pw& g) { return g.rows <= 16 ? 16 : g.rows <= 32 ? 32 : 64; }

template <typename T>
cudaError_t run_t(const Pw& g, int64_t ldx, const uint8_t* x, bool copied, const float* sx, const uint8_t* w, const float* sw,
                  const T* bias, T* y, cudaStream_t s) {
  if (plan(g) == Plan::Row) {
    switch (row_pixels(g)) {
      case 16: return launch_row<T, 16>(g, ldx, x, copied, sx, w, sw, bias, y, s);
      case 32: return launch_row<T, 32>(g, ldx, x, copied, sx, w, sw, bias, y, s);
      default: return launch_row<T, 64>(g, ldx, x, copied, sx, w, sw, bias, y, s);
    }
  }
  static std::atomic<uint64_t> ready_tile{0}, ready_pair{0};
  if (tiles_of(g, kM, Tile::kN) >= (int64_t(1) << 31)) return cudaErrorNotSupported;
  if (by_pairs(g)) return launch_tiles<Pair, T>(pair_kernel<T>, true, ready_pair, g, ldx, x, copied, sx, w, sw, bias, y, s);
  return launch_tiles<Tile, T>(tile_kernel<T>, false, ready_tile, g, ldx, x, copied, sx, w, sw, bias, y, s);
}

}  // namespace

// The row kernel up to 32 pixels, and while clusters of two and more find room
// and there is a long enough sum to share: 128 pixels, 4096 -> 4096 channels
// 11.6 us against 16.3 in tiles, 300, 4096 -> 512 8.6 against 16.2, 77, 1536 ->
// 1984 7.4 against 8.6; but 196, 512 -> 512 7.9 against 5.8.
Plan plan(const Pw& g) {
  const int np = row_pixels(g), split = split_of(g, np);
  if ((int64_t)((g.nkb + split - 1) / split) * np * 4 > 32 * 1024) return Plan::Tile;  // its table of scales
  return g.rows <= 32 || (g.nkb >= 10 && tiles_of(g, np, 128) <= 96) ? Plan::Row : Plan::Tile;
}

bool by_pairs(const Pw& g) {
  const int64_t tiles = tiles_of(g, kM, Tile::kN), pairs = tiles_of(g, 2 * kM, Pair::kN);
  // Measured: a call of tiles takes 2.9 us and per round 0.4 us a block of
  // channels and 1.35; a call of pairs (four times the products) 3.8, 0.6 and
  // 1.6. In tiles against pairs: 12544 pixels, 512 -> 512 channels 12.5 and
  // 13.8 us, 3136, 1024 -> 1024 12.2 and 10.9, 200704, 128 -> 128 22.3 and
  // 25.3, 10569, 2688 -> 1296 68.3 and 57.5, 8192, 4096 -> 4096 195 and 144.
  const int64_t by_tile = 2900 + (tiles + 151) / 152 * (g.nkb * 400 + 1350);
  const int64_t by_pair = 3800 + (pairs + 75) / 76 * (g.nkb * 600 + 1600);
  return by_pair < by_tile;
}

cudaError_t run_tc(const Pw& g, int64_t ldx, const uint8_t* x, bool copied, const float* sx, const uint8_t* w, const float* sw,
                   const void* bias, void* y, cudaStream_t s) {
  if (g.rows >= (int64_t(1) << 31) - 256) return cudaErrorNotSupported;  // coordinates of a copy are 32 bits
  cudaError_t e = cudaErrorInvalidValue;
  DWCONV_DISPATCH_DTYPE(g.dtype, T, e = run_t<T>(g, ldx, x, copied, sx, w, sw, (const T*)bias, (T*)y, s));
  return e;
}

}  // namespace pw8
}  // namespace dwconv
