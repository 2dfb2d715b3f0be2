// Slab and stream group-norm kernels, f16 instances.
#include "norm_slab_impl.cuh"

namespace dwconv {
namespace norm {
namespace slab {
template cudaError_t run_fwd<__half>(const Norm&, const Plan&, bool, const __half*, const __half*, const __half*, __half*, float*, float*,
                                 const Act8&, const Sums&, cudaStream_t);
template cudaError_t run_bwd<__half>(const Norm&, const Plan&, bool, const __half*, const Act8&, const __half*, const __half*, const __half*,
                                 const float*, const float*, __half*, const Sums&, cudaStream_t);
}  // namespace slab
}  // namespace norm
}  // namespace dwconv
