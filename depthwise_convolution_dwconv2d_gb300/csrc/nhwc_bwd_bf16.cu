// Row-walking channels-last backward, bf16 instances.
#include "nhwc_bwd_impl.cuh"

namespace dwconv {
namespace nhwc {
namespace walk {
template cudaError_t run<__nv_bfloat16>(const Conv&, const Geom&, bool, const __nv_bfloat16*, const Act8&, const __nv_bfloat16*, const __nv_bfloat16*, __nv_bfloat16*, float*,
                             cudaStream_t);
template cudaError_t run_staged<__nv_bfloat16>(const Conv&, const Staged&, int, const Views&, const Act8&, const __nv_bfloat16*, __nv_bfloat16*, float*,
                             cudaStream_t);
}  // namespace walk
}  // namespace nhwc
}  // namespace dwconv
