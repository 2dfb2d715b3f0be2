// RMS norm over the channels of a row, with the residual's addition and an
// output in 8 bits: geometry and entry points (rms.cu, rms_bwd.cu).
#pragma once

#include "act8.cuh"

namespace dwconv {
namespace rms {

// Validated geometry, passed to kernels by value.
struct Rms {
  int64_t rows;
  int C, dtype;
  float eps;
  int64_t xs, xo;  // distance of x's rows (residual, h, gx and their kind too), first channel
  int64_t ys, yo;  // the same of y and gy
};

// "row" (a row stays in the registers of its threads), "wide" (it is read
// twice) of pass 0 (forward) or 1 (backward), for aligned pointers
const char* plan_name(const Rms& g, int pass);
size_t bwd_workspace_bytes(const Rms& g);

// residual, gamma, h, y, rstd and t.codes may be null.
cudaError_t fwd(const Rms& g, const void* x, const void* residual, const void* gamma, void* h, void* y, float* rstd,
                const Act8& t, cudaStream_t s);
// gamma, gres, gx and ggamma may be null; ws only where ggamma is.
cudaError_t bwd(const Rms& g, const void* h, const void* gy, const void* gamma, const float* rstd, const void* gres,
                void* gx, void* ggamma, float* ws, cudaStream_t s);

// ---- how rows are laid over threads (rms.cu, rms_bwd.cu) --------------------
// tpr threads (a power of two) hold a row, each NI vectors of V channels.
// Neighbouring lanes hold neighbouring vectors, so that accesses are whole lines
// and a block of channels of a checkpoint stays within a warp; from item to
// item a thread goes on by tpr vectors (the forward that steps over rows) or by
// a warp's (the others).
struct Lay {
  int v;        // channels per vector: 16 bytes' worth, or 1
  int ni;       // vectors per thread
  int tpr;      // threads per row
  int nt;       // threads per block
  int segs;     // spans of tpr * ni vectors that a row takes: 1 keeps it in registers
};

inline int pow2_at_least(int64_t n) {
  int p = 1;
  while (p < n) p *= 2;
  return p;
}

}  // namespace rms
}  // namespace dwconv
