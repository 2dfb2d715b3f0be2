// Slab and stream group-norm kernels, f32 instances.
#include "norm_slab_impl.cuh"

namespace dwconv {
namespace norm {
namespace slab {
template cudaError_t run_fwd<float>(const Norm&, const Plan&, bool, const float*, const float*, const float*, float*, float*, float*,
                                 const Act8&, const Sums&, cudaStream_t);
template cudaError_t run_bwd<float>(const Norm&, const Plan&, bool, const float*, const Act8&, const float*, const float*, const float*,
                                 const float*, const float*, float*, const Sums&, cudaStream_t);
}  // namespace slab
}  // namespace norm
}  // namespace dwconv
