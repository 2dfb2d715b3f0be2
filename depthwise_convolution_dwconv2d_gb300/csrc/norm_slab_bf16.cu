// Slab and stream group-norm kernels, bf16 instances.
#include "norm_slab_impl.cuh"

namespace dwconv {
namespace norm {
namespace slab {
template cudaError_t run_fwd<__nv_bfloat16>(const Norm&, const Plan&, bool, const __nv_bfloat16*, const __nv_bfloat16*, const __nv_bfloat16*, __nv_bfloat16*, float*, float*,
                                 const Act8&, const Sums&, cudaStream_t);
template cudaError_t run_bwd<__nv_bfloat16>(const Norm&, const Plan&, bool, const __nv_bfloat16*, const Act8&, const __nv_bfloat16*, const __nv_bfloat16*, const __nv_bfloat16*,
                                 const float*, const float*, __nv_bfloat16*, const Sums&, cudaStream_t);
}  // namespace slab
}  // namespace norm
}  // namespace dwconv
