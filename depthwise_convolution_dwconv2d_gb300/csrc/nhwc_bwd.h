// Row-walking channels-last backward: shape support, plan and launch
// (nhwc_bwd.cu, nhwc_bwd_impl.cuh).
#pragma once

#include "act8.cuh"
#include "nhwc.h"

namespace dwconv {
namespace nhwc {

// Algo::Nhwc for the row-walking kernels, Algo::Generic otherwise.
Algo plan_bwd(const Conv& c);
size_t bwd_workspace_bytes(const Conv& c);
// gx [N, H, W, C], gw [C*m, kh, kw], gb [C*m], each or null; the input is x,
// or x8 where x is null.
cudaError_t bwd(const Conv& c, const void* x, const Act8& x8, const void* gy, const void* w, void* gx, void* gw,
                void* gb, bool accumulate, float* ws, cudaStream_t s);

namespace walk {

constexpr int kRingThreads = 256, kRingBlocks = 2;     // threads of a block, blocks per SM: 3x3 filters
constexpr int kBlockThreads = 128, kBlockBlocks = 2;   // 5x5 and 7x7

struct Geom {
  int64_t items;    // N * bands * strips
  int64_t groups;   // blocks' worth of items
  int ct_log;       // log2 of the channel pairs of a block's tile
  int tiles;        // channel tiles
  int chunks;       // blocks per channel tile = partial sums per filter value
  int strips;       // per row
  int bands;
  int band;         // gy rows of a band
  int t_begin, t_end;  // gy rows that the input's rows map to
  int v_begin;
  bool want_gx, want_gw, accumulate;
};

constexpr int kTileThreads = 128;
// Columns of a strip. A step is straight code, K * K * px * 2 / S packed
// products of it, and at 7x7 half as much of it pays: 5x45x51x96 fp32 22 us at
// eight columns, 17 at four; 22x147x17 of 55 samples 80 and 64; where blocks
// take many steps the repeated reads cost a little (32x28x28x128 bf16 31, 33).
// 5x5 at 32x28x28x128: 18.7 at eight, 20.7 at four.
constexpr int tile_px(int K) { return K == 7 ? 4 : 8; }

// The kernels that stage rows with the tensor memory accelerator: a block
// owns `cs` strips of `ns` samples, its lanes; a stage holds grows rows of gy
// and xrows of x per sample: as many as the register ring of the 3x3 kernel
// has, a whole band with the rows above it for the larger filters.
constexpr int kStagedThreads = 128;  // the most threads of a block
constexpr int kStagedBlocks = 4;     // blocks per SM
constexpr int kMaxStages = 4;
constexpr int kMostSmem = 208 * 1024;  // dynamic shared memory of a block at most
struct Staged {
  int ct_log, tiles, chunks;
  int strips, segs, cs, ns;
  int bands, band;
  int t_begin, t_end, v_begin;
  int items;           // per channel tile: sample groups * segs * bands, below 2^30
  FastDiv d_segs, d_bands;
  int threads;
  int stages;
  int grows, xrows;    // rows of a stage
  int gc, xc;          // columns of a stage's rows of gy and x
  int gy_bytes, x_bytes;      // of a stage's copies
  int x_at, stage_bytes;      // where x begins, and the next stage (multiples of 128)
  bool want_gx, want_gw, want_x, accumulate, pair_out;  // want_gw: gw or gb; want_x: gw; pair_out: two channels of gx are
                                                        // one aligned store
};

bool supported(const Conv& c);
Geom plan(const Conv& c);
// false: no staged form of this shape and source (kSrc*)
bool plan_staged(const Conv& c, int src, Staged* g);

// nhwc_bwd_{f32,f16,bf16}.cu. `pair`: two channels are one aligned access.
template <typename T>
cudaError_t run(const Conv& c, const Geom& g, bool pair, const T* x, const Act8& x8, const T* gy, const T* w, T* gx,
                float* ws, cudaStream_t s);
// gy (from its first channel) and x, or its codes, with the distance of their
// pixels in bytes.
struct Views {
  const void *gy, *x;
  int64_t gdist, xdist;
  bool copied;  // by a launch of this call
};
// cudaErrorNotSupported: a pointer or distance is no multiple of 16 bytes.
template <typename T>
cudaError_t run_staged(const Conv& c, const Staged& g, int src, const Views& v, const Act8& x8, const T* w, T* gx,
                       float* ws, cudaStream_t s);

}  // namespace walk
}  // namespace nhwc
}  // namespace dwconv
