// distill.cu -- distillation from a teacher's top logits: loss and gradient in one kernel.
//
// Per row of V student logits x with the teacher's logits t_k of the columns id_k (a negative id
// is no entry), z = scale * x, w the row's weight:
//   p_k = exp(scale t_k) / sum_k exp(scale t_k)     over the entries given,
//   log q_j = z_j - log sum_j exp z_j               over the whole row,
//   loss = w sum_k p_k (log p_k - log q_{id_k}),
//   dx_j = dloss w scale (q_j - sum_{k: id_k = j} p_k).
// Since the p_k add up to 1, with t* = max t_k, P = sum exp(scale (t_k - t*)) and the running sums
// of vocab.cuh about the reference r:
//   loss = w (scale sum_k p_k ((t_k - t*) - (x_{id_k} - r)) - log P + log Z).
#include <algorithm>
#include <math.h>

#include "distill_plan.h"
#include "vocab.cuh"
#include "vocab_ops.h"

namespace lnk {
namespace {

constexpr int kDsMaxWarps = 16;
constexpr int kDsMaxCluster = 8;
constexpr int kDsShare = LN_MAX_TOP / 32;  // a lane's entries of a teacher's list
constexpr int kDsTable = 8 * LN_MAX_TOP;

struct DsParams {
    const void* x;
    long long ld;
    const int* ids;
    const float* teacher;
    const float* weights;
    int rows;
    int V;
    int K;
    int staged;        // vectors of a slice that are kept in shared memory
    int chunk;         // vectors of one bulk copy
    int copies;        // of a slice, at most
    int blocks_shift;  // log2 of the blocks of a cluster
    float scale, c;    // c = scale * log2 e
    float dloss;
    float* losses;
    void* dx;
    long long ldd;
    unsigned* status;  // the per-device status word (bounded waits)
    uint64_t limit_ns;
};

// A row's teacher: made by one warp during the row before, but for x.
struct DsRow {
    int id[LN_MAX_TOP];
    float p[LN_MAX_TOP];
    float x[LN_MAX_TOP];  // the student's logit there, where this block has the column
    float w;       // the row's weight
    float co;      // dloss * w * scale: the factor of the gradient
    float spread;  // sum p (t - max t)
    float sum;     // sum exp(scale (t - max t))
    int learn;     // 0: no entry, or a row that does not count
    int bad;       // a column outside the row
    int twins;     // a column named twice
};

struct __align__(16) DsShared {
    uint64_t full[kDsSlots][kDsChunks];
    uint64_t met[2];  // the sums of a row have arrived from all blocks of the cluster
    DsRow row[3];  // the row before, whose list is still being written; this one; the next
    // Two of each, for rows in turn.  The sums (reference, z) of the warps of all blocks of the cluster.
    float2 total[2][kDsMaxCluster * kDsMaxWarps];
    // The blocks' entries, for the first block's loss: the largest of their x, sum p, sum p (x - largest).
    float4 list[2][kDsMaxCluster];
    int table[kDsTable];  // columns seen in a list
};

// A block's slice of a row: vectors [lo, hi), of which [lo, mid) are kept in shared memory.
template <typename T>
struct DsSlice {
    const T* xr;
    RowCut<T> cut;
    int lo, hi, mid;
    __device__ __forceinline__ DsSlice(const DsParams& p, int row, int rank)
        : xr(static_cast<const T*>(p.x) + (size_t)row * (size_t)p.ld), cut(xr, p.V) {
        const int per = (cut.nvec + (1 << p.blocks_shift) - 1) >> p.blocks_shift;
        lo = min(cut.nvec, rank * per);
        hi = min(cut.nvec, lo + per);
        mid = min(hi, lo + p.staged);
    }
    __device__ __forceinline__ const uint4* vectors() const {
        return reinterpret_cast<const uint4*>(xr + cut.head);
    }
    // Whether the block writes column j.
    __device__ __forceinline__ bool has(int j, int rank) const {
        const int in = j - cut.head, v = in / Io<T>::kVec;
        return in < 0 || v >= cut.nvec ? rank == 0 : v >= lo && v < hi;
    }
};

// The sums of all warps of the cluster joined, in the same order everywhere.
__device__ __forceinline__ RowTotal all_total(const float2* total, int n, float c) {
    RowTotal a{-INFINITY, 0.f, 0.f};
    for (int i = (int)threadIdx.x & 31; i < n; i += 32) a = total_join(a, {total[i].x, total[i].y, 0.f}, c);
    return warp_total(a, c);
}

// Rows are taken in turn by persistent blocks, or clusters of blocks that take a slice of the row
// each.  A slice comes into shared memory by bulk copies; NT threads sum it up chunk by chunk as it
// arrives, the warps exchange their sums (through the first of a row's two barriers), and form the
// gradient from shared memory: a row is read once.  The copies of the next row run meanwhile, so that
// neither the reductions nor the stores leave the memory without requests.  What does not fit
// (`staged`) is read a second time, through L2.
//
// What is not the row itself is the work of three more warps, beside the others': one starts the
// copies, forms the loss, and puts the gradient of the list's columns over what the others have
// written; one turns the next row's list into weights; one reads the logits of the list's columns.
// (As part of the other threads' work it made a row of 50304 take 6.7 us instead of 5.2.)
//
// Bound by the read and the write where a slice is kept whole and is not short: 8192 x 50304 bf16 with 64
// entries takes 273 us, 6.0 TB/s, 0.90 of what a copy gets (351 us with 256 entries: the list's warps set
// the pace).  A row's chain of meetings takes about 3 us whatever its length, which shows for rows of
// 32 KB (4000 x 16384: 54 us, 0.73).  Rows that do not fit are read again through L2, which also holds the
// gradient that is being written: 1024 x 131072 takes 111 us (0.72), split over clusters of four to keep
// all of it 112 us too, and over eight 230.
//
// WIDE: logits and gradient lie at the same place of a 16-byte vector in every row.
template <typename T, int NT, bool WIDE>
__global__ void __launch_bounds__(NT + 96, NT == 512 ? 1 : 2) distill_kernel(const DsParams p) {
    using IO = Io<T>;
    using PR = Pairs<T>;
    constexpr int kVec = IO::kVec;
    constexpr int H = PR::kPairs;
    constexpr int kStep = kBatch * NT;
    constexpr int kWarps = NT / 32;
    extern __shared__ __align__(128) unsigned char smem_raw[];
    __shared__ DsShared sh;
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int blocks = 1 << p.blocks_shift, rank = (int)blockIdx.x & (blocks - 1);
    const int first = (int)blockIdx.x >> p.blocks_shift, stride = (int)gridDim.x >> p.blocks_shift;
    const float nan = __int_as_float(0x7fc00000);
    // The meeting of a row: the sums of all warps are there.  Blocks of a cluster send theirs to one
    // another by asynchronous stores that an mbarrier of the receiver counts, not by the cluster's
    // barrier: its release would wait for the gradient of the row before to be written out.
    unsigned meetings = 0;
    auto meet = [&]() {
        if (blocks == 1) {
            __syncthreads();
            return true;
        }
        return mbar_wait(&sh.met[meetings & 1u], meetings >> 1 & 1u, p.limit_ns);
    };
    // A wait ran out somewhere in the block: what has been written is void, and the block ends with this
    // row -- going on, it would send the other blocks of its cluster sums that they do not wait for yet.
    bool dead = false;

    // The mbarriers and the first list are there, in all blocks of the cluster.
    auto begin = [&]() {
        __syncthreads();
        if (blocks > 1) {
            cluster_arrive();
            cluster_wait();
        }
    };
    // No block ends before what the others send it has arrived.
    auto end_together = [&]() {
        if (blocks > 1) {
            cluster_arrive();
            cluster_wait();
        }
    };
    // A row of weight 0 is not read.
    auto weight = [&](int row) { return row >= p.rows ? 0.f : p.weights ? p.weights[row] : 1.f; };

    if (warp == kWarps) {
        // ---- The warp that starts the copies and finishes the rows.
        SlotPhases started;
        auto issue = [&](int row, int slot) {  // lane 0
            const DsSlice<T> g(p, row, rank);
            unsigned char* to = smem_raw + 16 * (size_t)(slot * p.staged);
            int i = 0;
            for (int v = g.lo; v < g.mid; ++i, v += p.chunk) {
                const unsigned bytes = 16u * (unsigned)(min(g.mid, v + p.chunk) - v);
                mbar_arrive_expect_tx(&sh.full[slot][i], bytes);
                bulk_g2s(to + 16 * (size_t)(v - g.lo), g.vectors() + v, bytes, &sh.full[slot][i]);
            }
            // Every row arms all of the plan's copies (SlotPhases), with nothing where its slice ends before.
            for (; i < p.copies; ++i) mbar_arrive(&sh.full[slot][i]);
            started.used(slot);
        };
        if (lane == 0) {
            for (int i = 0; i < kDsSlots * kDsChunks; ++i) mbar_init(&sh.full[0][0] + i, 1);
            mbar_init(&sh.met[0], 1);
            mbar_init(&sh.met[1], 1);
            fence_barrier_init();
        }
        pdl_enter();
        const float w = weight(first), w1 = weight(first + stride);
        if (lane == 0) {
            if (w != 0.f) issue(first, 0);
            if (w1 != 0.f) issue(first + stride, 1);
        }
        begin();
        for (int row = first, slot = 0, n = 0; row < p.rows; row += stride, slot ^= 1, n = n == 2 ? 0 : n + 1) {
            const float w2 = weight(row + 2 * stride);
            const DsRow& q = sh.row[n];
            const bool learn = q.learn;
            RowTotal a{0.f, 1.f, 0.f};
            float r = 0.f;
            bool gone = false;
            if (learn) {
                const int turn = (int)(meetings & 1u);
                if (blocks > 1 && lane == 0)
                    mbar_arrive_expect_tx(&sh.met[turn], (unsigned)blocks * kWarps * 8u +
                                                             16u * (rank == 0 ? (unsigned)blocks : 1u));
                gone = !meet();
                ++meetings;
                a = all_total(sh.total[turn], blocks * kWarps, p.c);
                r = a.ref == -INFINITY ? 0.f : a.ref;
                if (rank == 0 && lane == 0 && p.losses) {
                    float gap = 0.f;
                    for (int i = 0; i < blocks; ++i) {
                        const float4 l = sh.list[turn][i];
                        gap += fmaf(l.x - r, l.y, l.z);
                    }
                    p.losses[row] = q.bad ? nan
                                          : q.w * (fmaf(q.spread - gap, p.scale, -logf(q.sum)) + logf(a.z));
                }
            } else if (rank == 0 && lane == 0 && p.losses) {
                p.losses[row] = 0.f;
            }
            dead = __syncthreads_or(gone);  // the slice is written, its slot free, the next list ready
            if (dead) break;
            if (lane == 0 && w2 != 0.f) issue(row + 2 * stride, slot);
            if (learn && p.dx) {
                const DsSlice<T> g(p, row, rank);
                T* dr = static_cast<T*>(p.dx) + (size_t)row * (size_t)p.ldd;
                const float cz = q.co / a.z;
                for (int k = lane; k < p.K; k += 32) {
                    const int j = q.id[k];
                    if (j < 0 || j >= p.V || !g.has(j, rank)) continue;
                    float sum = q.p[k];
                    bool only = true;
                    if (q.twins) {
                        // One writer a column: the first of the entries that name it, with all their
                        // weights.
                        sum = 0.f;
                        for (int i = 0; i < p.K; ++i) {
                            if (q.id[i] != j) continue;
                            if (i < k) only = false;
                            sum += q.p[i];
                        }
                    }
                    if (only) dr[j] = IO::from_f(fmaf(ex2_fast((q.x[k] - r) * p.c), cz, -q.co * sum));
                }
                __syncwarp();
            }
        }
        if (dead && lane == 0) {
            raise_status(p.status, kStatusTimeout);
            for (int slot = 0; slot < kDsSlots; ++slot)  // copies still in flight
                for (int i = 0; i < p.copies; ++i)
                    (void)mbar_wait(&sh.full[slot][i], started.parity(slot) ^ 1u, p.limit_ns);
        }
        end_together();
        return;
    }

    if (warp == kWarps + 1) {
        // ---- The warp that gets the lists ready.
        pdl_enter();
        int id[kDsShare];
        float t[kDsShare], w = 0.f;
        auto load_list = [&](int row) {
            w = weight(row);
#pragma unroll
            for (int j = 0; j < kDsShare; ++j) {
                if (32 * j >= p.K) break;
                const int k = lane + 32 * j;
                id[j] = -1;
                t[j] = -INFINITY;
                if (k < p.K && row < p.rows) {
                    id[j] = p.ids[(size_t)row * p.K + k];
                    t[j] = p.teacher[(size_t)row * p.K + k];
                }
            }
        };
        auto prepare = [&](DsRow& q) {
            float most = -INFINITY;
            bool odd = false, bad = false;
#pragma unroll
            for (int j = 0; j < kDsShare; ++j) {
                if (32 * j >= p.K) break;
                if (id[j] < 0) continue;
                bad |= id[j] >= p.V;
                odd |= t[j] != t[j];
                most = fmaxf(most, t[j]);
            }
            // Columns named twice: each entry looks for its own in a table of many times the list's
            // size, left empty again.
            int at[kDsShare], found[kDsShare];
#pragma unroll
            for (int j = 0; j < kDsShare; ++j) {
                if (32 * j >= p.K) break;
                at[j] = (int)(((unsigned)id[j] * 0x9e3779b1u) >> 21);
                found[j] = id[j] >= 0 ? atomicCAS(&sh.table[at[j]], -1, id[j]) : -1;
            }
            static_assert(kDsTable == 2048, "the hash above has 11 bits");
            most = warp_max(most);
            bad = __any_sync(kFullMask, bad);
            odd = __any_sync(kFullMask, odd);
            float e[kDsShare], sum = 0.f, spread = 0.f, zero = 0.f;
#pragma unroll
            for (int j = 0; j < kDsShare; ++j) {
                if (32 * j >= p.K) break;
                e[j] = id[j] >= 0 ? ex2_fast((t[j] - most) * p.c) : 0.f;
                sum += e[j];
            }
            warp_sum2(sum, zero);
#pragma unroll
            for (int j = 0; j < kDsShare; ++j) {
                if (32 * j >= p.K) break;
                const int k = lane + 32 * j;
                if (k >= p.K) continue;
                const float pk = e[j] / sum;
                q.id[k] = id[j];
                q.p[k] = pk;
                if (pk != 0.f) spread += pk * (t[j] - most);
            }
            warp_sum2(spread, zero);
            bool twin = false;
#pragma unroll
            for (int j = 0; j < kDsShare; ++j) {
                if (32 * j >= p.K) break;
                while (found[j] != -1 && found[j] != id[j]) {  // another column has the place
                    at[j] = (at[j] + 1) % kDsTable;
                    found[j] = atomicCAS(&sh.table[at[j]], -1, id[j]);
                }
                twin |= found[j] != -1;
            }
            twin = __any_sync(kFullMask, twin);  // (and every entry has its place)
#pragma unroll
            for (int j = 0; j < kDsShare; ++j) {
                if (32 * j >= p.K) break;
                if (id[j] >= 0) sh.table[at[j]] = -1;
            }
            if (lane == 0) {
                q.w = w;
                q.co = bad ? nan : p.dloss * w * p.scale;
                q.spread = spread;
                q.sum = sum;
                q.learn = w != 0.f && (most != -INFINITY || odd || bad);
                q.bad = bad;
                q.twins = twin;
            }
            __syncwarp();
        };
        for (int i = lane; i < kDsTable; i += 32) sh.table[i] = -1;
        __syncwarp();
        load_list(first);
        prepare(sh.row[0]);
        load_list(first + stride);
        begin();
        for (int row = first, n = 0; row < p.rows; row += stride) {
            const bool learn = sh.row[n].learn;
            n = n == 2 ? 0 : n + 1;
            if (row + stride < p.rows) {
                prepare(sh.row[n]);
                load_list(row + 2 * stride);
            }
            if (learn && blocks == 1) meet();
            if (__syncthreads_or(0)) break;
        }
        end_together();
        return;
    }

    if (warp == kWarps + 2) {
        // ---- The warp that reads the logits of the list's columns.
        pdl_enter();
        begin();
        SlotPhases phases;
        for (int row = first, slot = 0, n = 0; row < p.rows; row += stride, slot ^= 1, n = n == 2 ? 0 : n + 1) {
            DsRow& q = sh.row[n];
            bool gone = false;
            if (q.w != 0.f) {
                const DsSlice<T> g(p, row, rank);
                const T* xs = reinterpret_cast<const T*>(smem_raw + 16 * (size_t)(slot * p.staged));
                for (int i = 0, v = g.lo; v < g.mid; ++i, v += p.chunk)
                    gone |= !mbar_wait(&sh.full[slot][i], phases.parity(slot), p.limit_ns);
                phases.used(slot);
                if (q.learn) {
                    // The student's logits at the list's columns, and this block's part of the loss about
                    // the largest of them.  An entry of weight 0 adds nothing, whatever the student has
                    // there; -inf elsewhere makes the loss infinite.
                    float x[kDsShare], most = -INFINITY;
#pragma unroll
                    for (int j = 0; j < kDsShare; ++j) {
                        if (32 * j >= p.K) break;
                        const int k = lane + 32 * j;
                        x[j] = -INFINITY;
                        if (k >= p.K) continue;
                        const int c = q.id[k];
                        if (c < 0 || c >= p.V || !g.has(c, rank)) continue;
                        const int in = c - g.cut.head, v = in / kVec;
                        x[j] = IO::to_f(in >= 0 && v < g.mid ? xs[in - g.lo * kVec] : g.xr[c]);
                        q.x[k] = x[j];
                        if (q.p[k] != 0.f) most = fmaxf(most, x[j]);
                    }
                    most = warp_max(most);
                    if (most == -INFINITY) most = 0.f;
                    float mass = 0.f, gap = 0.f;
#pragma unroll
                    for (int j = 0; j < kDsShare; ++j) {
                        if (32 * j >= p.K) break;
                        const int k = lane + 32 * j;
                        if (k >= p.K) continue;
                        const int c = q.id[k];
                        const float pk = q.p[k];
                        if (c < 0 || c >= p.V || pk == 0.f || !g.has(c, rank)) continue;
                        mass += pk;
                        gap += pk * (x[j] - most);
                    }
                    warp_sum2(mass, gap);
                    const int turn = (int)(meetings & 1u);
                    if (lane == 0) {
                        float4* l = &sh.list[turn][rank];
                        if (blocks == 1) *l = make_float4(most, mass, gap, 0.f);
                        if (blocks > 1) send4(in_block(l, 0), most, mass, gap, in_block(&sh.met[turn], 0));
                        // The other blocks' own meetings wait for it too: the logits that it has read may
                        // be overwritten then.
                        if (rank > 0)
                            send4(in_block(l, (uint32_t)rank), most, mass, gap, in_block(&sh.met[turn], (uint32_t)rank));
                    }
                    if (blocks == 1) meet();
                    ++meetings;
                }
            }
            if (__syncthreads_or(gone)) break;
        }
        end_together();
        return;
    }

    // ---- The warps that sum up the rows and write the gradient.
    pdl_enter();
    const f2 c2 = f2_splat(p.c);
    SlotPhases phases;
    // The part of a slice that is not kept, a batch in flight while the one before is dealt with.
    auto each_batch = [&](const DsSlice<T>& g, auto deal) {
        const uint4* xv = g.vectors();
        int v0 = g.mid + tid;
        if (v0 >= g.hi) return;
        uint4 a[kBatch], b[kBatch];
        load_batch<T>(a, xv, v0, NT, g.hi);
        while (true) {
            load_batch<T>(b, xv, v0 + kStep, NT, g.hi);
            deal(a, v0);
            if ((v0 += kStep) >= g.hi) break;
            load_batch<T>(a, xv, v0 + kStep, NT, g.hi);
            deal(b, v0);
            if ((v0 += kStep) >= g.hi) break;
        }
    };
    begin();
    for (int row = first, slot = 0, n = 0; row < p.rows; row += stride, slot ^= 1, n = n == 2 ? 0 : n + 1) {
        const DsSlice<T> g(p, row, rank);
        const DsRow& q = sh.row[n];
        const uint4* xs = reinterpret_cast<const uint4*>(smem_raw) + (size_t)slot * p.staged;
        T* dr = p.dx ? static_cast<T*>(p.dx) + (size_t)row * (size_t)p.ldd : nullptr;
        const bool has_loose = rank == 0 && tid < g.cut.nloose();
        const bool learn = q.learn;
        const int end = g.mid - g.lo;
        bool gone = false;
        RowSums<false> s;
        s.clear();
        if (q.w != 0.f) {
            // Pass 1: the slice's sums.
            for (int i = 0, from = 0; from < end; ++i, from += p.chunk) {
                gone |= !mbar_wait(&sh.full[slot][i], phases.parity(slot), p.limit_ns);
                if (!learn) continue;
                const int to = min(end, from + p.chunk);
                for (int v0 = from + tid; v0 < to; v0 += kStep) {
                    uint4 u[kBatch];
                    if (v0 + (kBatch - 1) * NT < to) {
#pragma unroll
                        for (int k = 0; k < kBatch; ++k) u[k] = xs[v0 + k * NT];
                    } else {
#pragma unroll
                        for (int k = 0; k < kBatch; ++k)
                            u[k] = v0 + k * NT < to ? xs[v0 + k * NT] : no_logits<T>();
                    }
                    if (s.see_batch<T>(u, p.c) > -INFINITY)
                        s.add_batch<T>(u, c2);
                }
            }
            phases.used(slot);
        }
        if (learn) {
            each_batch(g, [&](const uint4 (&u)[kBatch], int) {
                if (s.see_batch<T>(u, p.c) > -INFINITY)
                    s.add_batch<T>(u, c2);
            });
            const float xl = has_loose ? IO::to_f(g.xr[g.cut.loose(tid)]) : 0.f;
            if (has_loose) s.add_one(xl, p.c);
            RowTotal a = warp_total({s.ref, f2_lo(s.z2) + f2_hi(s.z2), 0.f}, p.c);
            const int turn = (int)(meetings & 1u);
            float2* mine = &sh.total[turn][rank * kWarps + warp];
            if (blocks > 1) {
                if (lane < blocks)
                    send2(in_block(mine, (uint32_t)lane), a.ref, a.z, in_block(&sh.met[turn], (uint32_t)lane));
            } else if (lane == 0) {
                *mine = make_float2(a.ref, a.z);
            }
            gone |= !meet();
            ++meetings;
            a = all_total(sh.total[turn], blocks * kWarps, p.c);
            if (dr) {
                // Pass 2: the gradient.
                const float r = a.ref == -INFINITY ? 0.f : a.ref;
                const float cz = q.co / a.z;
                const f2 cz2 = f2_splat(cz);
                auto put = [&](const uint4& u, T* to) {
                    f2 o[H];
                    less<T>(u, r, o);
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        const f2 z = f2_mul(o[h], c2);
                        o[h] = f2_mul(f2_make(ex2_fast(f2_lo(z)), ex2_fast(f2_hi(z))), cz2);
                    }
                    if constexpr (WIDE) {
                        st_stream(to, PR::pack(o));
                    } else {
#pragma unroll
                        for (int h = 0; h < H; ++h) {
                            to[2 * h] = IO::from_f(f2_lo(o[h]));
                            to[2 * h + 1] = IO::from_f(f2_hi(o[h]));
                        }
                    }
                };
                T* to = dr + g.cut.col(g.lo + tid);
                int v = tid;
                for (; v + (kBatch - 1) * NT < end; v += kStep, to += kStep * kVec) {
#pragma unroll
                    for (int k = 0; k < kBatch; ++k) put(xs[v + k * NT], to + k * NT * kVec);
                }
                for (; v < end; v += NT, to += NT * kVec) put(xs[v], to);
                each_batch(g, [&](const uint4 (&u)[kBatch], int v0) {
                    T* at = dr + g.cut.col(v0);
#pragma unroll
                    for (int k = 0; k < kBatch; ++k)
                        if (v0 + k * NT < g.hi) put(u[k], at + k * NT * kVec);
                });
                if (has_loose) dr[g.cut.loose(tid)] = IO::from_f(ex2_fast((xl - r) * p.c) * cz);
            }
        } else if (dr) {
            if constexpr (WIDE) {
                for (int v = g.lo + tid; v < g.hi; v += NT) st_stream(dr + g.cut.col(v), make_uint4(0, 0, 0, 0));
            } else {
                for (int j = g.cut.col(g.lo) + tid; j < g.cut.col(g.hi); j += NT) dr[j] = IO::from_f(0.f);
            }
            if (has_loose) dr[g.cut.loose(tid)] = IO::from_f(0.f);
        }
        if (__syncthreads_or(gone)) break;
    }
    end_together();
}

// ---------------------------------------------------------------------------------------
// Short rows (a batch a thread): one row a block, the row in the threads' registers, many blocks an
// SM.  A row is little work, so what counts is that many are under way; the copies and extra warps of
// the kernel above take longer than the row does (8192 rows of 1024 bf16 logits, 64 entries: 46 us there,
// 17 here, 2.2 TB/s; bound by the chain of a row's steps).
// ---------------------------------------------------------------------------------------
template <typename T, int NT, bool WIDE>
__global__ void __launch_bounds__(NT, 1024 / NT) distill_short_kernel(const DsParams p) {
    using IO = Io<T>;
    using PR = Pairs<T>;
    constexpr int kVec = IO::kVec;
    constexpr int H = PR::kPairs;
    constexpr int kWarps = NT / 32;
    constexpr int kTable = NT < LN_MAX_TOP ? 4 * NT : 4 * LN_MAX_TOP;
    __shared__ __align__(16) int sh_id[LN_MAX_TOP];
    __shared__ float sh_t[LN_MAX_TOP];
    __shared__ int sh_table[kTable];  // columns seen in the list
    __shared__ RowTotal sh_total[kWarps];
    __shared__ float sh_gap[kWarps];
    const int tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float nan = __int_as_float(0x7fc00000);
    pdl_enter();
    const size_t row = blockIdx.x;
    const float w = p.weights ? p.weights[row] : 1.f;
    const T* xr = static_cast<const T*>(p.x) + row * (size_t)p.ld;
    T* dr = p.dx ? static_cast<T*>(p.dx) + row * (size_t)p.ldd : nullptr;
    const RowCut<T> cut(xr, p.V);
    const uint4* xv = reinterpret_cast<const uint4*>(xr + cut.head);
    const bool has_loose = tid < cut.nloose();
    uint4 u[kBatch];
    float xl = 0.f;
    if (w != 0.f) {  // a row of weight 0 is not read
        load_batch<T>(u, xv, tid, NT, cut.nvec);
        if (has_loose) xl = IO::to_f(xr[cut.loose(tid)]);
    }
    int id = -1;  // the list's entry k is thread k's (there are no more entries than threads)
    float t = -INFINITY, x = 0.f;
    if (tid < p.K) {
        id = p.ids[row * p.K + tid];
        if (id >= 0) t = p.teacher[row * p.K + tid];
        if (w != 0.f && id >= 0 && id < p.V) x = IO::to_f(xr[id]);
        sh_id[tid] = id;
        sh_t[tid] = t;
    }
    for (int i = tid; i < kTable; i += NT) sh_table[i] = -1;
    __syncthreads();
    // Every warp sums the list up for itself.
    float most = -INFINITY;
    bool bad = false, odd = false;
    for (int k = lane; k < p.K; k += 32) {
        bad |= sh_id[k] >= p.V;
        odd |= sh_t[k] != sh_t[k];
        most = fmaxf(most, sh_t[k]);
    }
    most = warp_max(most);
    bad = __any_sync(kFullMask, bad);
    odd = __any_sync(kFullMask, odd);
    if (w == 0.f || (most == -INFINITY && !odd && !bad)) {
        if (tid == 0 && p.losses) p.losses[row] = 0.f;
        if (dr) {
            if constexpr (WIDE) {
                for (int v = tid; v < cut.nvec; v += NT) st_stream(dr + cut.col(v), make_uint4(0, 0, 0, 0));
                if (has_loose) dr[cut.loose(tid)] = IO::from_f(0.f);
            } else {
                for (int j = tid; j < p.V; j += NT) dr[j] = IO::from_f(0.f);
            }
        }
        return;
    }
    float sum = 0.f, zero = 0.f;
    for (int k = lane; k < p.K; k += 32)
        if (sh_id[k] >= 0) sum += ex2_fast((sh_t[k] - most) * p.c);
    warp_sum2(sum, zero);
    RowSums<false> s;
    s.clear();
    const f2 c2 = f2_splat(p.c);
    if (tid < cut.nvec && s.see_batch<T>(u, p.c) > -INFINITY)
        s.add_batch<T>(u, c2);
    if (has_loose) s.add_one(xl, p.c);
    RowTotal a = warp_total({s.ref, f2_lo(s.z2) + f2_hi(s.z2), 0.f}, p.c);
    if (lane == 0) sh_total[warp] = a;
    // A column named twice: each entry looks for its own in a table four times the list's size.
    bool twin = false;
    float pk = 0.f;
    if (id >= 0) {
        pk = ex2_fast((t - most) * p.c) / sum;
        unsigned at = ((unsigned)id * 0x9e3779b1u >> 22) % kTable;
        while (true) {
            const int old = atomicCAS(&sh_table[at], -1, id);
            twin = old == id;
            if (old == -1 || twin) break;
            at = (at + 1) % kTable;
        }
    }
    __syncthreads();
    a = lane < kWarps ? sh_total[lane] : RowTotal{-INFINITY, 0.f, 0.f};
    a = warp_total(a, p.c);
    const float r = a.ref == -INFINITY ? 0.f : a.ref;
    if (p.losses) {
        // An entry of weight 0 adds nothing, whatever the student has there.
        float gap = pk != 0.f ? pk * ((t - most) - (x - r)) : 0.f;
        warp_sum2(gap, zero);
        if (lane == 0) sh_gap[warp] = gap;
    }
    const float co = bad ? nan : p.dloss * w * p.scale, cz = co / a.z;
    if (dr) {
        const f2 cz2 = f2_splat(cz);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int v = tid + k * NT;
            if (v >= cut.nvec) break;
            f2 o[H];
            less<T>(u[k], r, o);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const f2 z = f2_mul(o[h], c2);
                o[h] = f2_mul(f2_make(ex2_fast(f2_lo(z)), ex2_fast(f2_hi(z))), cz2);
            }
            T* to = dr + cut.col(v);
            if constexpr (WIDE) {
                st_stream(to, PR::pack(o));
            } else {
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    to[2 * h] = IO::from_f(f2_lo(o[h]));
                    to[2 * h + 1] = IO::from_f(f2_hi(o[h]));
                }
            }
        }
        if (has_loose) dr[cut.loose(tid)] = IO::from_f(ex2_fast((xl - r) * p.c) * cz);
    }
    twin = __syncthreads_or(twin);  // the row is written; the warps' parts of the loss
    if (tid == 0 && p.losses) {
        float gap = 0.f;
        for (int i = 0; i < kWarps; ++i) gap += sh_gap[i];
        p.losses[row] = bad ? nan : w * (fmaf(gap, p.scale, -logf(sum)) + logf(a.z));
    }
    if (!dr || id < 0 || id >= p.V) return;
    // One writer a column: the first of the entries that name it, with all their weights.
    if (twin) {
        pk = 0.f;
        for (int k = 0; k < p.K; ++k) {
            if (sh_id[k] != id) continue;
            if (k < tid) return;
            pk += ex2_fast((sh_t[k] - most) * p.c) / sum;
        }
    }
    dr[id] = IO::from_f(fmaf(ex2_fast((x - r) * p.c), cz, -co * pk));
}

template <typename T, int NT>
const void* distill_short_variant(bool wide) {
    return wide ? (const void*)distill_short_kernel<T, NT, true> : (const void*)distill_short_kernel<T, NT, false>;
}

template <typename T, int NT>
const void* distill_variant(bool wide) {
    return wide ? (const void*)distill_kernel<T, NT, true> : (const void*)distill_kernel<T, NT, false>;
}

template <typename T>
cudaError_t launch_distill_t(const DistillArgs& a, cudaStream_t stream) {
    constexpr int kVec = Io<T>::kVec;
    DsParams p;
    p.x = a.logits;
    p.ld = a.ld;
    p.ids = a.ids;
    p.teacher = a.teacher;
    p.weights = a.weights;
    p.V = a.V;
    p.K = a.K;
    p.scale = a.scale;
    p.c = a.scale * kLog2e;
    p.dloss = a.dloss;
    p.losses = a.losses;
    p.dx = a.dlogits;
    p.ldd = a.ldd;
    p.status = a.status;
    p.limit_ns = a.wait_limit_ns;
    p.rows = a.rows;
    const int nvec = a.V / kVec, sms = device_info(-1).sms;
    const bool wide = !a.dlogits || rows_congruent(a.logits, a.ld, a.dlogits, a.ldd, sizeof(T), a.rows);
    void* args[] = {&p};
    if (nvec <= 1024 || (nvec <= 512 * kBatch && a.rows <= 2 * sms)) {
        int nt = 64;
        while (nt * kBatch < nvec || nt < a.K) nt *= 2;
        const void* kern = nt == 64    ? distill_short_variant<T, 64>(wide)
                           : nt == 128 ? distill_short_variant<T, 128>(wide)
                           : nt == 256 ? distill_short_variant<T, 256>(wide)
                                       : distill_short_variant<T, 512>(wide);
        return launch_kernel(kern, dim3((unsigned)a.rows), dim3(nt), 0, stream, args, false);
    }
    const DistillPlan plan = distill_plan(a.rows, nvec, sms, kBatch);
    static_assert(kDsMaxCluster == 8, "distill_plan goes up to 8 blocks");
    const int blocks = plan.blocks, nt = plan.threads;
    p.blocks_shift = blocks == 8 ? 3 : blocks == 4 ? 2 : blocks == 2 ? 1 : 0;
    p.staged = plan.staged;
    p.chunk = plan.chunk;
    p.copies = plan.copies;
    const size_t smem = (size_t)kDsSlots * p.staged * 16;
    const void* kern = nt == 512 ? distill_variant<T, 512>(wide) : distill_variant<T, 256>(wide);
    const cudaError_t e = allow_smem(kern, smem);
    if (e != cudaSuccess) return e;
    const int at_once = clusters_at_once(kern, nt + 96, blocks, smem);
    if (at_once < 1) return cudaErrorInvalidConfiguration;
    return launch_cluster(kern, dim3((unsigned)(std::min(a.rows, at_once) * blocks)), dim3(nt + 96), blocks, smem,
                          stream, args);
}

}  // namespace

cudaError_t launch_distill(Dtype dt, const DistillArgs& a, cudaStream_t stream, int* launches) {
    cudaError_t e = dt == Dtype::F32 ? launch_distill_t<float>(a, stream)
                                     : launch_distill_t<__nv_bfloat16>(a, stream);
    *launches = e == cudaSuccess;
    return e;
}

}  // namespace lnk
