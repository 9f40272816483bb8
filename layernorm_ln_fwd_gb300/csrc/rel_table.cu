// rel_table.cu -- the softmax with a relative position bias: which kernel takes a call, and the second stage of
// the table's gradient.  Each block of the backward left its dS by bucket, a row of partial sums for each head
// that it worked on; block k's of head h is row k + h, since either grows by one at a time along the blocks' units.
// Here a head's rows are added: 16 interleaved groups, then the groups, in order, with the rounding errors of the
// additions carried along.
#include <algorithm>

#include "ln_finish.cuh"
#include "rel_ops.h"

namespace lnk {
namespace {

constexpr int kTabX = 32, kTabY = 16;

template <typename T>
__global__ void __launch_bounds__(kTabX * kTabY) rel_table_kernel(const float* part, T* dtable, int H, int blocks,
                                                                  int64_t per_head, int total) {
    __shared__ float2 fold[kTabY][kTabX];
    pdl_enter();
    const int h = blockIdx.x, k = (int)blockIdx.y * kTabX + (int)threadIdx.x;
    // The blocks that have units of the head: block b has those from units b / blocks on.
    const int64_t units = per_head * H, u0 = per_head * h, u1 = u0 + per_head;
    auto block_of = [&](int64_t u) {  // the last block that begins at unit u or before
        int64_t b = min(u * blocks / units, (int64_t)blocks - 1);
        while (b + 1 < blocks && units * (b + 1) / blocks <= u) ++b;
        return (int)b;
    };
    const int b0 = block_of(u0), b1 = block_of(u1 - 1);
    float s = 0.f, c = 0.f;
    if (k < total)
#pragma unroll 4
        for (int b = b0 + (int)threadIdx.y; b <= b1; b += kTabY) comp_add(s, c, part[(int64_t)(b + h) * total + k], 0.f);
    fold[threadIdx.y][threadIdx.x] = make_float2(s, c);
    __syncthreads();
    if (threadIdx.y == 0 && k < total) {
        for (int g = 1; g < kTabY; ++g) comp_add(s, c, fold[g][threadIdx.x].x, fold[g][threadIdx.x].y);
        // (a sum that is not finite has no meaningful error term)
        dtable[(int64_t)k * H + h] = Io<T>::from_f(fabsf(s) < INFINITY ? s + c : s);
    }
}

}  // namespace

void rel_span(const RelArgs& a, int* dlo, int* dhi) {
    // At least one distance on each side that has buckets of its own, so that each has its far end.
    const int last = a.buckets->n ? a.buckets->edge[a.buckets->n - 1] : 1;
    *dlo = -last;
    *dhi = a.buckets->both ? last : 0;
    if (!a.q_pos) {  // positions 0 .. Lq - 1: distances beyond these do not occur
        *dlo = std::max(*dlo, -(a.Lq - 1));
        *dhi = std::min(*dhi, a.Lk - 1);
    }
}

// Few queries a sequence over short rows: a warp a row, one row a block, where there are rows enough for all SMs and the
// window is one that a warp fills in time; else a block a row, which fills it 8 times as fast.  bf16, one query, 128
// distances, a warp and a block a row: 96 rows of 210 keys 4.7 and 3.4 us, 1024 of 502 5.2 and 6.4, 8192 of 502 11 and
// 28; with 800 distances 96 rows of 210 14.7 and 4.6.
constexpr int kRelNarrow = 300;
bool rel_single(int Lq, int nvec, int span, int64_t rows) {
    return Lq < 4 && nvec <= 64 && span <= kRelNarrow && rows > 4 * (int64_t)device_info(-1).sms;
}

// Rows of up to 512 vectors go to teams of 4 vectors a lane, several teams a block, so that a block has several rows on
// their way and only a row's own warps wait for one another; parts of a warp where a row has no use for one.  bf16,
// 12 heads, forward / backward with the table's gradient, us, beside another shape's:
//   128 x 128 (x 256 sequences)        8 lanes x 2 37 / 57      a warp x 1                 109 / 123
//   256 x 256 (x 64)                   16 lanes x 2 36 / 57     a warp x 1                 51 / 64
//   512 x 512 (x 16)                   16 lanes x 4 34.5 / 57   a warp x 2                 37 / 57
//   1024 x 1024 (x 4)                  a warp x 4 35 / 59       8 warps x 1                114 / 103
//   2048 x 2048 (x 2)                  2 warps x 4 72 / 108     8 warps x 1                135 / 127
//   4096 x 4096                        4 warps x 4 144 / 204    8 warps x 2                172 / 189
//   the last, causal                                122 / 145                              152 / 157
// The backward's full rows beyond 384 vectors alone go to 8 warps (8 and 4 warps: 288 vectors 83 and 74 us, 320 94 and 84, 360
// 112 and 101; 400 131 and 120, 448 152 and 148, so that the border could lie higher; 512 189 and 204).  Four vectors a lane take 80
// registers, three blocks an SM (rel_resident): held to 64 they spill, and the same take 34.5 -> 38, 35 -> 40, 72 -> 80.
int rel_shape(int V, int64_t rows, int Lq, int Lk, int span, bool bwd, bool causal, bool* slots) {
    const int nvec = (Lk + V - 1) / V;
    auto fits = [&](int teams) { return rel_slot_count(teams) * rel_groups(span, V) * V * 4 <= kRelSlotBytes; };
    *slots = nvec <= 2048 && fits(8);
    if (*slots && rel_single(Lq, nvec, span, rows)) return 9;
    if (*slots && Lq >= 4 && nvec <= (bwd && !causal ? 384 : 512)) {
        if (nvec <= 16 && fits(32)) return nvec <= 8 ? 10 : 11;
        if (nvec <= 64 && fits(16)) return nvec <= 32 ? 12 : 13;
        return nvec <= 32 ? 5 : nvec <= 64 ? 6 : nvec <= 128 ? 7 : nvec <= 256 ? 8 : 14;
    }
    return nvec <= 256 ? 0 : nvec <= 512 ? 1 : nvec <= 1024 ? 2 : nvec <= 2048 ? 3 : 4;
}

// The same for shifted rows (bf16, 12 heads, 501 x 501 x 16: parts of a warp 44 us forward, a warp 56; 4001 x 4001: 4
// warps 190 / 212, 8 warps 219 / 242).  In the backward a warp holds a row at least: parts of one would take too many
// slots.  In bf16 rows of up to 32 vectors are better moved, by parts of a warp (32 heads, shifted and moved: 32 x
// 65 x 65 49 and 35 us, 16 x 138 x 138 causal 49 and 42, 16 x 201 x 201 66 and 61, 8 x 283 x 283 causal 57 and 56, 8 x 501 x
// 501 causal 93 and 104; fp32 16 x 101 x 101 28 and 28, 8 x 201 x 201 37 and 46).
int rel_shape_shifted(int V, int64_t rows, int Lq, int Lk, int span, bool bwd, int* copies) {
    if (bwd && V == 8 && Lk <= 32 * V) return -1;
    const int nvec = (Lk + V - 1 + V - 1) / V;  // chunks that a row may lie in
    int shape = nvec <= 256 ? 0 : nvec <= 512 ? 1 : nvec <= 1024 ? 2 : nvec <= 2048 ? 3 : -1;
    if (rel_single(Lq, nvec, span, rows)) shape = 9;
    if (Lq >= 4 && nvec <= 512) shape = nvec <= 32 ? 5 : nvec <= 64 ? 6 : nvec <= 128 ? 7 : nvec <= 256 ? 8 : 14;
    if (!bwd && Lq >= 4 && nvec <= 64) {
        const int parts = nvec <= 16 ? (nvec <= 8 ? 10 : 11) : nvec <= 32 ? 12 : 13;
        if (rel_slot_count(kRelShapes[parts].teams) * rel_groups(span, V) * V * 4 <= kRelSlotBytes) shape = parts;
    }
    if (shape < 0) return -1;
    const int teams = kRelShapes[shape].teams;
    *copies = bwd ? teams * V : rel_slot_count(teams);
    return *copies * rel_groups(span, V) * V * 4 <= (bwd ? kRelShiftedBytes : kRelSlotBytes) ? shape : -1;
}

size_t rel_workspace_bytes(int H, int buckets, int sms) {
    return ((size_t)kRelMaxPerSm * sms + (size_t)H) * (size_t)buckets * sizeof(float);
}

cudaError_t launch_rel_table(const RelArgs& a, int blocks, int64_t per_head, cudaStream_t stream) {
    int total = (a.buckets->n + 1) * (a.buckets->both ? 2 : 1);
    const float* part = a.part;
    int H = a.H;
    const dim3 grid(H, (total + kTabX - 1) / kTabX), block(kTabX, kTabY);
    void* out = a.dtable;
    void* args[] = {&part, &out, &H, &blocks, &per_head, &total};
    const void* kern = a.table_f32 ? (const void*)rel_table_kernel<float> : (const void*)rel_table_kernel<__nv_bfloat16>;
    return launch_kernel(kern, grid, block, 0, stream, args, false);
}

}  // namespace lnk
