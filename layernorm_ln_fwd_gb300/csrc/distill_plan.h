// distill_plan.h -- how the distillation kernel's rows are cut into blocks and copies, and the phases of
// the copies' mbarriers.  Plain C++ apart from the marks of what the device calls too, so that the
// arithmetic is checked on the host for other numbers of SMs.
#pragma once

#include <algorithm>

#ifdef __CUDACC__
#define LNK_BOTH __host__ __device__ __forceinline__
#else
#define LNK_BOTH inline
#endif

namespace lnk {

constexpr int kDsChunks = 8;  // bulk copies of a row's slice
constexpr int kDsSlots = 2;   // rows a block holds: the one it works on and the next
constexpr int kDsRoom = 100 * 64;  // vectors of a slot at most: two slots, and a block an SM

struct DistillPlan {
    int blocks;   // of a cluster: a row's slices
    int threads;  // that sum up the rows
    int staged;   // vectors of a slice that are kept in shared memory
    int chunk;    // vectors of one bulk copy: whole batches of the block
    int copies;   // of a slice, at most
};

// For rows of `nvec` vectors (one fewer where a row starts inside a vector); `batch`: vectors of a thread
// that are loaded together.
inline DistillPlan distill_plan(int rows, int nvec, int sms, int batch) {
    DistillPlan p;
    // Blocks of a cluster: where there are fewer rows than SMs, as many as keep them all busy; and where
    // far more of a row than a slot would be read again.
    p.blocks = 1;
    while (p.blocks < 8 && (nvec / p.blocks > 11 * kDsRoom / 4 ||
                            ((long long)rows * p.blocks * 2 <= sms && nvec / (p.blocks * 2) >= 512)))
        p.blocks *= 2;
    // A row a little too long for a slot goes to two blocks where that leaves less of the last round idle:
    // 512 x 65536 bf16 takes 7 rounds of half rows, 31.6 us, for 4 of whole ones, 35.0 (where both come out
    // alike, one block: 300 x 65536 20.2 us, 21.7 in two).
    if (p.blocks == 1 && nvec > kDsRoom && nvec <= 2 * kDsRoom) {
        const int ones = (rows + sms - 1) / sms, twos = (rows + sms / 2 - 1) / (sms / 2);
        if (10 * twos < 18 * ones) p.blocks = 2;
    }
    const int slice = std::max(1, (nvec + p.blocks - 1) / p.blocks);
    p.threads = slice > 36 * 64 ? 512 : 256;
    p.staged = std::min(slice, kDsRoom);
    const int all = p.threads * batch;
    p.chunk = ((p.staged + 3) / 4 + all - 1) / all * all;
    p.copies = (p.staged + p.chunk - 1) / p.chunk;
    return p;
}

// The phase that the next row's copies into each slot complete.  One bit for all copies of a slot does,
// since every row that is read arms all of the plan's copies: rows of an odd distance differ by a vector
// (1025 vectors are two copies of 1024, 1024 are one), and an mbarrier that one row of a slot left
// out would be a phase behind for the next.
struct SlotPhases {
    unsigned bits = 0;
    LNK_BOTH unsigned parity(int slot) const { return bits >> slot & 1u; }
    LNK_BOTH void used(int slot) { bits ^= 1u << slot; }
};

}  // namespace lnk
