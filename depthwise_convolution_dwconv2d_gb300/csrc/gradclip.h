// Norm over all gradients of a model and their clipping (gradclip.cu).
#pragma once

#include "common.cuh"

namespace dwconv {
namespace clip {

size_t workspace_bytes(int count, const dwconv_grad_t* grads);
// Validated tensors; most is +infinity for no clipping. norm may be null.
cudaError_t run(int count, const dwconv_grad_t* grads, float most, float* norm, void* ws, cudaStream_t s);

}  // namespace clip
}  // namespace dwconv
