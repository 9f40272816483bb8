// rel_fwd_bf16.cu -- Forward kernels of the softmax with a relative position bias, bf16.
#include "rel_softmax.cuh"

namespace lnk {

cudaError_t launch_rel_fwd_bf16(const RelArgs& a, cudaStream_t stream, int* launches) {
    return launch_rel_t<__nv_bfloat16, false>(a, stream, launches);
}

}  // namespace lnk
