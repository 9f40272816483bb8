// rel_bwd_f32.cu -- Backward kernels of the softmax with a relative position bias, fp32.
#include "rel_softmax.cuh"

namespace lnk {

cudaError_t launch_rel_bwd_f32(const RelArgs& a, cudaStream_t stream, int* launches) {
    return launch_rel_t<float, true>(a, stream, launches);
}

}  // namespace lnk
