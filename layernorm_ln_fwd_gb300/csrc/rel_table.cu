// rel_table.cu -- the softmax with a relative position bias: how a call's rows are cut, and the second stage
// of the table's gradient: each block of the backward left its dS by bucket, one row of partial sums; here
// those of a head are added, 16 interleaved groups of rows and then the groups, in a fixed order, with the
// rounding errors of the additions carried along (their number grows with the batch).
#include <algorithm>

#include "ln_finish.cuh"
#include "rel_ops.h"

namespace lnk {
namespace {

constexpr int kTabX = 32, kTabY = 16;

template <typename T>
__global__ void __launch_bounds__(kTabX * kTabY) rel_table_kernel(const float* part, T* dtable, int H, int B,
                                                                  int chunks, int total) {
    __shared__ float2 fold[kTabY][kTabX];
    pdl_enter();
    const int h = blockIdx.x, k = (int)blockIdx.y * kTabX + (int)threadIdx.x;
    float s = 0.f, c = 0.f;
    if (k < total) {
        const int64_t n = (int64_t)B * chunks;
#pragma unroll 4
        for (int64_t i = threadIdx.y; i < n; i += kTabY) {
            const int64_t b = i / chunks;
            comp_add(s, c, part[((b * H + h) * chunks + (i - b * chunks)) * total + k], 0.f);
        }
    }
    fold[threadIdx.y][threadIdx.x] = make_float2(s, c);
    __syncthreads();
    if (threadIdx.y == 0 && k < total) {
        for (int g = 1; g < kTabY; ++g) comp_add(s, c, fold[g][threadIdx.x].x, fold[g][threadIdx.x].y);
        // (a sum that is not finite has no meaningful error term)
        dtable[(int64_t)k * H + h] = Io<T>::from_f(fabsf(s) < INFINITY ? s + c : s);
    }
}

}  // namespace

RelPlan rel_plan(Dtype dt, int64_t matrices, int Lq, int Lk, int sms) {
    // Shapes of kRelShapes (rel_softmax.cuh) by the vectors of a row.
    const int nvec = (Lk + (dt == Dtype::F32 ? 4 : 8) - 1) / (dt == Dtype::F32 ? 4 : 8);
    RelPlan p;
    int teams = 1;
    if (Lq < 4 && nvec <= 512) {  // single queries: a block each, no teams to fill
        p.shape = nvec <= 64 ? 8 : nvec <= 256 ? 9 : 10;
    } else if (nvec <= 128) {
        p.shape = nvec <= 32 ? 0 : nvec <= 64 ? 1 : 2;
        teams = 8;
    } else if (nvec <= 512) {
        p.shape = nvec <= 256 ? 3 : 4;
        teams = nvec <= 256 ? 4 : 2;
    } else {
        p.shape = nvec <= 1024 ? 5 : nvec <= 2048 ? 6 : 7;
    }
    // Enough blocks to even out their ends, rows enough for a block to pay for its window.
    int64_t rows = matrices * Lq / ((int64_t)sms * 16);
    rows = std::min<int64_t>(std::max<int64_t>(rows, 1), 128);
    rows = (rows + teams - 1) / teams * teams;
    p.chunks = (int)((Lq + rows - 1) / rows);
    p.rows = (Lq + p.chunks - 1) / p.chunks;
    p.rows = (p.rows + teams - 1) / teams * teams;
    p.chunks = (Lq + p.rows - 1) / p.rows;
    return p;
}

size_t rel_workspace_bytes(Dtype dt, int64_t matrices, int Lq, int Lk, int buckets, int sms) {
    return (size_t)matrices * (size_t)rel_plan(dt, matrices, Lq, Lk, sms).chunks * (size_t)buckets * sizeof(float);
}

cudaError_t launch_rel_table(const RelArgs& a, const RelPlan& plan, cudaStream_t stream) {
    int total = (a.buckets->n + 1) * (a.buckets->both ? 2 : 1);
    const float* part = a.part;
    int H = a.H, B = a.B, chunks = plan.chunks;
    const dim3 grid(H, (total + kTabX - 1) / kTabX), block(kTabX, kTabY);
    void* out = a.dtable;
    void* args[] = {&part, &out, &H, &B, &chunks, &total};
    const void* kern = a.table_f32 ? (const void*)rel_table_kernel<float> : (const void*)rel_table_kernel<__nv_bfloat16>;
    return launch_kernel(kern, grid, block, 0, stream, args, false);
}

}  // namespace lnk
