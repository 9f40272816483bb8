// vocab_ops.h -- host-side declarations of the operators over rows of logits (logprobs.cu, distill.cu)
// and of what their launches need beside ln_internal.h's.
#pragma once

#include "ln_internal.h"

namespace lnk {

// Clusters of `blocks` blocks (1: blocks) of a kernel that run on the current device at once,
// cached.
int clusters_at_once(const void* kern, int threads, int blocks, size_t smem);

// Lets `kern` have `bytes` of dynamic shared memory on the current device (asked of the driver only
// when it is more than before).
cudaError_t allow_smem(const void* kern, size_t bytes);

// launch_kernel with clusters of `blocks` blocks along the grid (1: none; up to 8).
cudaError_t launch_cluster(const void* kern, dim3 grid, dim3 block, int blocks, size_t smem,
                           cudaStream_t stream, void** args);

// Token log probabilities with entropy, rank and top alternatives (null outputs are left out;
// `tokens` null: no logp and no ranks; `top` 0: no alternatives).
struct LogprobsArgs {
    const void* logits;
    int64_t ld;
    const int* tokens;
    int rows;
    int V;
    float scale;
    int top;
    float* logp;
    float* entropy;
    float* lse;
    int* ranks;
    int* top_ids;
    float* top_logp;
};

cudaError_t launch_logprobs(Dtype dt, const LogprobsArgs& a, cudaStream_t stream, int* launches);

// Their gradient (dlogp or dentropy may be null; dlogits may alias logits).
struct LogprobsBwdArgs {
    const void* logits;
    int64_t ld;
    const int* tokens;
    const float* lse;
    const float* entropy;
    const float* dlogp;
    const float* dentropy;
    int rows;
    int V;
    float scale;
    void* dlogits;
    int64_t ldd;
};

cudaError_t launch_logprobs_bwd(Dtype dt, const LogprobsBwdArgs& a, cudaStream_t stream,
                                int* launches);

// Distillation from a teacher's top logits: losses (optional) and dlogits (optional; may alias
// logits).
struct DistillArgs {
    const void* logits;
    int64_t ld;
    const int* ids;
    const float* teacher;
    const float* weights;
    int rows;
    int V;
    int K;
    float scale;
    float dloss;
    float* losses;
    void* dlogits;
    int64_t ldd;
    unsigned* status;  // the per-device status word (bounded waits)
    uint64_t wait_limit_ns;
};

cudaError_t launch_distill(Dtype dt, const DistillArgs& a, cudaStream_t stream, int* launches);

// Whether rows of `lda` elements at a and of `ldb` at b start at the same place of a 16-byte vector,
// every row of them.
bool rows_congruent(const void* a, int64_t lda, const void* b, int64_t ldb, size_t esize, int rows);

}  // namespace lnk
