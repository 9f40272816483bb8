// rel_fwd_f32.cu -- Forward kernels of the softmax with a relative position bias, fp32.
#include "rel_softmax.cuh"

namespace lnk {

cudaError_t launch_rel_fwd_f32(const RelArgs& a, cudaStream_t stream, int* launches) {
    return launch_rel_t<float, false>(a, stream, launches);
}

}  // namespace lnk
