// Channels-last group norm with an activation: geometry and entry points
// (norm.cu).
#pragma once

#include "act8.cuh"

namespace dwconv {
namespace norm {

// Validated geometry, passed to kernels by value. Rows are pixels.
struct Norm {
  int64_t N, P;       // samples, pixels of a sample
  int C, G, D;        // channels, groups, channels per group
  int act, dtype;
  float eps;
  int64_t xs, xo;     // distance of x's rows, first channel
  int64_t ys, yo;     // the same of y
};

// "slab", "stream" or "split"; a function of the descriptor alone
const char* plan_name(const Norm& g, int pass);
size_t workspace_bytes(const Norm& g, int pass);

// x8.codes == nullptr: no checkpoint.
cudaError_t fwd(const Norm& g, const void* x, const void* gamma, const void* beta, void* y, float* mean,
                float* rstd, float* ws, const Act8& x8, cudaStream_t s);
// x == nullptr: the input is x8.
cudaError_t bwd(const Norm& g, const void* x, const Act8& x8, const void* gy, const void* gamma,
                const void* beta, const float* mean, const float* rstd, void* gx, void* ggamma, void* gbeta,
                float* ws, cudaStream_t s);

}  // namespace norm
}  // namespace dwconv
