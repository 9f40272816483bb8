// rel_bwd_bf16.cu -- Backward kernels of the softmax with a relative position bias, bf16.
#include "rel_softmax.cuh"

namespace lnk {

cudaError_t launch_rel_bwd_bf16(const RelArgs& a, cudaStream_t stream, int* launches) {
    return launch_rel_t<__nv_bfloat16, true>(a, stream, launches);
}

}  // namespace lnk
