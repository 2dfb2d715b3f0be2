// Row-walking channels-last backward: shape support, plan and launch
// (nhwc_bwd.cu, nhwc_bwd_impl.cuh).
#pragma once

#include "nhwc.h"

namespace dwconv {
namespace nhwc {
namespace walk {

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

bool supported(const Conv& c);
Geom plan(const Conv& c);

// nhwc_bwd_{f32,f16,bf16}.cu. `pair`: two channels are one aligned access.
template <typename T>
cudaError_t run(const Conv& c, const Geom& g, bool pair, const T* x, const Act8& x8, const T* gy, const T* w, T* gx,
                float* ws, cudaStream_t s);

}  // namespace walk
}  // namespace nhwc
}  // namespace dwconv
