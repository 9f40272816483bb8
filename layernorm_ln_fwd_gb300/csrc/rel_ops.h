// rel_ops.h -- host-side declarations of the softmax with a relative position bias (rel_*.cu) and of the
// 8-bit checkpoints (ckpt8.cu, ckpt8_norm.cu).
#pragma once

#include "vocab_ops.h"

namespace lnk {

constexpr int kRelMaxEdges = 255;

// The bias's buckets: bucket(d) for d = key - query is the number of edges at or below |d| (0 for a key behind
// its query where `both` is false), plus edges + 1 for d > 0 where it is true.
struct RelBuckets {
    int n;      // edges
    int both;
    int edge[kRelMaxEdges];
};

struct RelArgs {
    const void* a;            // scores (forward) or dy (backward)
    const void* y;            // backward: probabilities, or null with q and k
    void* out;                // y (forward) or dx (backward)
    int64_t lda, ldy, ldo;    // elements between rows
    int8_t* q;                // checkpoint: integers [rows, whole blocks] and bytes [rows, blocks], or null
    uint8_t* k;
    const void* mask;         // additive [mask_rows, Lk], or null
    int64_t mask_rows;
    const void* table;        // [buckets, H]
    bool table_f32;           // fp32, or bf16
    const int* lens;          // [B] keys of each sequence, or null
    const int* q_pos;         // [B] position of each sequence's first query, or null
    int B, H, Lq, Lk;
    bool causal;
    float scale;
    const RelBuckets* buckets;
    void* dtable;             // backward: [buckets, H] of the table's type, or null
    float* part;              // its partial sums (rel_workspace_bytes)
};

constexpr int kRelFar = 1 << 30;  // positions are held to this: every bucket ends long before

// Lanes of a row, rows of a block at a time, vectors a lane; rows of any length in tiles, twice.
struct RelShape {
    int lanes, teams, nv;
    bool loop;
};
constexpr RelShape kRelShapes[] = {{256, 1, 1, false}, {256, 1, 2, false}, {256, 1, 4, false}, {512, 1, 4, false},
                                   {512, 1, 4, true}, {32, 8, 1, false}, {32, 8, 2, false}, {32, 8, 4, false},
                                   {64, 4, 4, false}, {32, 1, 2, false}, {8, 32, 1, false}, {8, 32, 2, false},
                                   {16, 16, 2, false}, {16, 16, 4, false}, {128, 2, 4, false}};
constexpr int kRelShapeCount = sizeof(kRelShapes) / sizeof(kRelShapes[0]);

// The window in shared memory as slots (rel_softmax.cuh): how many, and groups of V entries of each.
__host__ __device__ constexpr int rel_slot_count(int teams) { return teams > 8 ? teams : 8; }
__host__ __device__ constexpr int rel_groups(int span, int V) { return (span - 1 + 2 * V - 1 + V - 1) / V + 1; }
// Bytes of all slots at most.  bf16, 12 heads, 16 x 512 x 512 with 400 distances a side, in slots and with what fits in 24 KB:
// forward 35.7 and 37.8 us, backward 58 and 61; 4 x 1024 x 1024 with 800 36 and 157 (one window), 64 and 170.  64 KB measures
// the same up to there.
constexpr int kRelSlotBytes = 48 * 1024;
// In the backward of shifted rows, with slots for each team: 32, 64, 96 KB (the window that does not fit is moved rows'),
// 4 x 1001 x 1001 with 150 distances a side 86, 70, 70 us, with 250 92, 92, 79; 16 x 501 x 501 with 150 92, 84, 84, with 250
// 96, 96, 103.
constexpr int kRelShiftedBytes = 64 * 1024;

constexpr int kRelMaxPerSm = 8;  // resident blocks of any shape that a launch uses

// The distances a call's window has to hold.
void rel_span(const RelArgs& a, int* dlo, int* dhi);
// The kernel's shape, and whether its window is in slots, for vectors of V elements.
int rel_shape(int V, int64_t rows, int Lq, int Lk, int span, bool bwd, bool causal, bool* slots);

// The shape for shifted rows and the slots that it has, or -1.
int rel_shape_shifted(int V, int64_t rows, int Lq, int Lk, int span, bool bwd, int* copies);

// Bytes of partial sums: a row of buckets for each block and head that it works on.
size_t rel_workspace_bytes(int H, int buckets, int sms);

cudaError_t launch_rel_fwd_f32(const RelArgs& a, cudaStream_t stream, int* launches);
cudaError_t launch_rel_fwd_bf16(const RelArgs& a, cudaStream_t stream, int* launches);
cudaError_t launch_rel_bwd_f32(const RelArgs& a, cudaStream_t stream, int* launches);
cudaError_t launch_rel_bwd_bf16(const RelArgs& a, cudaStream_t stream, int* launches);
// The second stage of the table's gradient, behind `blocks` blocks of the first.
cudaError_t launch_rel_table(const RelArgs& a, int blocks, int64_t per_head, cudaStream_t stream);

// x [rows, cols], rows ld elements apart, to integers and bytes, and back (into rows ld apart).
cudaError_t launch_ckpt8_store(Dtype dt, const void* x, int64_t ld, int64_t rows, int cols, int8_t* q,
                               uint8_t* k, cudaStream_t stream);
cudaError_t launch_ckpt8_load(Dtype dt, const int8_t* q, const uint8_t* k, int64_t rows, int cols, void* x,
                              int64_t ld, cudaStream_t stream);

// The LayerNorm's (mean given) or RMSNorm's backward from a checkpoint of its input.
struct CkptNormArgs {
    const void* dy;
    const int8_t* q;
    const uint8_t* k;
    const void* gamma;
    const float* mean;   // null: RMSNorm
    const float* rstd;
    void* dx;
    void* dgamma;
    void* dbeta;
    int rows, cols;
    float* part;         // ckpt_norm_workspace_bytes
};
size_t ckpt_norm_workspace_bytes(int rows, int cols, bool rms, int sms);
cudaError_t launch_ckpt_norm_bwd(Dtype dt, const CkptNormArgs& a, cudaStream_t stream, int* launches);

}  // namespace lnk
