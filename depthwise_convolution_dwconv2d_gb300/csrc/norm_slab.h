// Slab and stream kernels of the channels-last group norm: plan and launch
// (norm_slab_impl.cuh, norm_slab_{f32,f16,bf16}.cu).
#pragma once

#include "norm.h"

namespace dwconv {
namespace norm {
namespace slab {

constexpr int kNT = 256;
constexpr int kMostSmem = 220 * 1024;  // dynamic shared memory of a block at most
constexpr int kMaxParts = 256;  // chunks of a stream
constexpr int kBatch = 4;  // rows that a thread fetches at a time; the next batch is on its way

// How a thread's V channels lie: side by side, one access of V elements; or a
// row's vectors apart, V accesses of one element each (for distances and
// pointers that rule the wide access out).
struct Plan {
  int V;
  bool strided;
  int S;           // channels of a slice (the last slice may have fewer)
  int vpr;         // vectors of a slice's row, idle lanes included
  int rl;          // row lanes: kNT / vpr
  int slices;
  int groups;      // groups of a slice
  int parts;       // blocks of a sample's slice: a cluster (slab), or chunks of pixels (stream)
  int rows;        // pixels of a block
  FastDiv d_vpr, d_slices, d_parts, d_D;
  float total, inv_total, inv_D;   // values of a (sample, group), and reciprocals
  int data_bytes;  // shared memory for a slab block's share of the inputs, a stream block's two batches
};

// Shared memory behind the shares: the row lanes' sums, tables per channel
// and per group.
inline int scratch_bytes(const Plan& k, int pass) {
  return (kNT * 2 * k.V + k.vpr * (pass ? 2 : 3) * k.V) * 4 + 2 * k.groups * 8;
}

// What passes between the kernels of a call, in its workspace: per (sample,
// part, group) the forward's (mean, squares) or the backward's (s1, s2), per
// (sample, part, channel) the backward's (sum du, sum du * xh). A slab has
// one part.
struct Sums {
  float2 *groups, *channels;
};

// slab = true: one launch of clusters; false: sums, then outputs.
template <typename T>
cudaError_t run_fwd(const Norm& g, const Plan& k, bool slab, const T* x, const T* gamma, const T* beta, T* y,
                    float* mean, float* rstd, const Act8& x8, const Sums& sums, cudaStream_t s);
template <typename T>
cudaError_t run_bwd(const Norm& g, const Plan& k, bool slab, const T* x, const Act8& x8, const T* gy, const T* gamma,
                    const T* beta, const float* mean, const float* rstd, T* gx, const Sums& sums, cudaStream_t s);

}  // namespace slab
}  // namespace norm
}  // namespace dwconv
