// Slab kernels of the channels-last group norm: plan and launch
// (norm_slab_impl.cuh, norm_slab_{f32,f16,bf16}.cu).
#pragma once

#include "norm.h"

namespace dwconv {
namespace norm {
namespace slab {

constexpr int kNT = 256;

struct Plan {
  int S;           // channels of a slice (the last slice may have fewer)
  int vpr;         // vectors of a slice's row, a block's idle lanes included
  int rl;          // row lanes: kNT / vpr
  int slices;
  int cl;          // blocks of a cluster
  int rows;        // pixels of a block's share
  int groups;      // groups of a slice
  int data_bytes;  // shared memory for the shares
};

// Shared memory behind the shares: the row lanes' sums, tables per channel
// and per group.
inline int scratch_bytes(const Plan& k, int V, int pass) {
  const int np = (V + 1) / 2;
  return (kNT * 4 * np + k.vpr * 4 * np + (pass ? 0 : k.vpr * 2 * np)) * 4 + 2 * k.groups * 8;
}

// Sums per (sample, channel) of the backward go to sums[N][C].
template <typename T>
cudaError_t run_fwd(const Norm& g, const Plan& k, int V, const T* x, const T* gamma, const T* beta, T* y, float* mean,
                    float* rstd, const Act8& x8, cudaStream_t s);
template <typename T>
cudaError_t run_bwd(const Norm& g, const Plan& k, int V, const T* x, const Act8& x8, const T* gy, const T* gamma,
                    const T* beta, const float* mean, const float* rstd, T* gx, float2* sums, cudaStream_t s);

}  // namespace slab
}  // namespace norm
}  // namespace dwconv
