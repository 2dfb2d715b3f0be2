// Row-walking channels-last backward, f16 instances.
#include "nhwc_bwd_impl.cuh"

namespace dwconv {
namespace nhwc {
namespace walk {
template cudaError_t run<__half>(const Conv&, const Geom&, bool, const __half*, const Act8&, const __half*, const __half*, __half*, float*,
                             cudaStream_t);
template cudaError_t run_staged<__half>(const Conv&, const Staged&, int, const Views&, const Act8&, const __half*, __half*, float*,
                             cudaStream_t);
}  // namespace walk
}  // namespace nhwc
}  // namespace dwconv
