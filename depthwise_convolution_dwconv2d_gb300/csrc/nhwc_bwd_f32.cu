// Row-walking channels-last backward, f32 instances.
#include "nhwc_bwd_impl.cuh"

namespace dwconv {
namespace nhwc {
namespace walk {
template cudaError_t run<float>(const Conv&, const Geom&, bool, const float*, const Act8&, const float*, const float*, float*, float*,
                             cudaStream_t);
template cudaError_t run_staged<float>(const Conv&, const Staged&, int, const Views&, const Act8&, const float*, float*, float*,
                             cudaStream_t);
}  // namespace walk
}  // namespace nhwc
}  // namespace dwconv
