// logprobs.cu -- log probabilities of given tokens over rows of logits, with the entropy, the
// token's rank and the top alternatives, and the gradient of the log probability and the entropy.
//
// Per row of V logits x with token t, z = scale * x:
//   L = log sum_j exp z_j,  q_j = exp(z_j - L),  logp = z_t - L,  H = -sum_j q_j log q_j,
//   dx_j = scale (dlogp (1[j = t] - q_j) - dH q_j (log q_j + H)).
// With u = (x - r) scale log2 e about a reference r (vocab.cuh), Z = sum 2^u and W = sum 2^u u:
//   L = scale r + log Z,   log q_j = (x_j - r) scale - log Z,   H = log Z - ln 2 W / Z.
#include <algorithm>
#include <math.h>

#include "top_select.cuh"
#include "vocab.cuh"
#include "vocab_ops.h"

namespace lnk {
namespace {

constexpr int kLpMaxThreads = 256;  // four such blocks an SM, of 64 registers a thread
constexpr int kLpSegments = 2048;   // segments of a slice at most, about
constexpr int kLpCand = 512;        // candidates held at once
constexpr int kLpCount = 128;       // entries that are put in order by counting
constexpr int kLpFlagged = 2 * LN_MAX_TOP;
constexpr int kLpLoose = 32;        // more than the loose elements of a row cut at 32 bytes
constexpr int kLpMaxCluster = 8;

struct LpParams {
    const void* x;
    long long ld;
    const int* tokens;
    int V;
    int top;
    int seg_shift;  // log2 of the vectors of a thread that share a segment: whole batches, or one vector (0)
    int nt_shift;   // log2 of the block's threads
    int nseg;       // segments: a multiple of the block's threads
    float scale, c;  // c = scale * log2 e
    float* logp;
    float* entropy;
    float* lse;
    int* ranks;
    int* top_ids;
    float* top_logp;
};

struct TopShared {
    SelectShared sel;
    entry_t cand[kLpCand];
    int flagged[kLpFlagged];
    int nflag, ncand;
    // entry_t sorted[max(kLpCand, blocks * top)], in a cluster entry_t joined[blocks * top], and
    // unsigned segs[nseg + kLpLoose] follow
};

// What a block of a cluster hands to the first.
struct LpShare {
    RowTotal total;
    int above;
};

// The top entries of a slice of a row whose segments' largest values are in `segs`.
//
// While the row streams by, nothing is done for the top but to keep the largest value of each
// segment (a few batches of one thread), a value the running sums need anyway.  The k-th largest
// of these is a lower bound of the k-th largest element: k different segments hold an element that
// is as large.  So only segments whose largest value reaches the bound can hold a top element -- k
// of them, or a few more for a bound found with some slack -- and those alone are read again (from
// L2: the row has just been read), their elements that reach the bound becoming the candidates.
//
// Where the candidates do not fit (many equal values at the bound: a constant row, a row masked by
// the type's lowest value; or few segments that hold very many large ones), the k-th largest entry
// of those that did fit is a bound as well, a higher one and one between columns of the same value.
// Each such round leaves out all but k of the kLpCand that were held, so the rounds end.
//
// Returns the number of candidates in sh->cand (in no order), all of the top among them; at most
// kLpCand.
template <typename T>
__device__ __forceinline__ int collect_top(const LpParams& p, const uint4* xv, int lo, int hi,
                                           const RowCut<T, 32>& cut, TopShared* sh, const unsigned* segs) {
    using IO = Io<T>;
    constexpr int kVec = IO::kVec;
    const int tid = (int)threadIdx.x, nt = (int)blockDim.x, k = p.top;
    const int nall = p.nseg + kLpLoose;
    // Vector i of a segment, counted from the slice's first.
    auto vector_of = [&](int seg, int i) {
        const int f = (seg >> p.nt_shift << p.seg_shift) + i;  // of the thread's vectors
        return pair_vector(2 * (seg & (nt - 1)) + nt * (f & ~(kBatch - 1)), nt, f & (kBatch - 1));
    };
    // Every element of the bound's value, whatever its column.
    entry_t bound = (entry_t)select_threshold(segs, nall, k, k / 4 + 16, &sh->sel) << 32;
    while (true) {
        const unsigned reach = (unsigned)(bound >> 32);  // the same for segments: values alone
        const float least = reach <= 1 ? -3.402823466e38f : order_value(reach);
        if (tid == 0) sh->nflag = sh->ncand = 0;
        __syncthreads();
#pragma unroll 1
        for (int i = tid; i < nall; i += nt) {
            const unsigned key = segs[i];
            if (key == 0 || key < reach) continue;
            if (i >= p.nseg) {  // a loose element
                const entry_t e = (entry_t)key << 32 | (uint32_t)~(uint32_t)cut.loose(i - p.nseg);
                if (e < bound) continue;
                const int at = atomicAdd(&sh->ncand, 1);
                if (at < kLpCand) sh->cand[at] = e;
                continue;
            }
            // A segment of the bound's value has nothing behind the bound's column.
            if (key == reach && (unsigned)cut.col(lo + vector_of(i, 0)) > ~(unsigned)bound) continue;
            if (*(volatile int*)&sh->nflag > kLpFlagged) continue;  // too many to list
            const int at = atomicAdd(&sh->nflag, 1);
            if (at < kLpFlagged) sh->flagged[at] = i;
        }
        __syncthreads();
        const bool listed = sh->nflag <= kLpFlagged;  // else all segments are gone through
        const int items = (listed ? sh->nflag : p.nseg) << p.seg_shift;
#pragma unroll 1
        for (int w0 = tid; w0 < items; w0 += kBatch * nt) {
            if (*(volatile int*)&sh->ncand > kLpCand) break;  // another round anyway
            uint4 u[kBatch];
            int col[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int w = w0 + b * nt;
                u[b] = no_logits<T>();
                if (w >= items) continue;
                const int q = w >> p.seg_shift, i = w & ((1 << p.seg_shift) - 1);
                const int seg = listed ? sh->flagged[q] : q;
                const unsigned key = segs[seg];
                const int v = lo + vector_of(seg, i);
                col[b] = cut.col(v);
                if (v >= hi || key < reach || (key == reach && (unsigned)col[b] > ~(unsigned)bound)) continue;
                u[b] = __ldcg(xv + v);
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (!(vector_max<T>(u[b]) >= least)) continue;
                float f[kVec];
                IO::unpack(u[b], f);
                unsigned take = 0;
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    take |= (unsigned)(f[j] >= least && make_entry(f[j], col[b] + j) >= bound) << j;
                if (take == 0) continue;
                int at = atomicAdd(&sh->ncand, __popc(take));
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    if (take >> j & 1u) {
                        if (at < kLpCand) sh->cand[at] = make_entry(f[j], col[b] + j);
                        ++at;
                    }
            }
        }
        __syncthreads();
        const int n = sh->ncand;
        if (n <= kLpCand) return n;
        bound = select_threshold(sh->cand, kLpCand, k, k / 2, &sh->sel);
    }
}

// The top of `list` in order into `out`; returns how many there are.
__device__ __forceinline__ int put_in_order(const entry_t* list, int n, int k, entry_t* sorted,
                                            TopShared* sh, entry_t** out) {
    if (n <= kLpCount) {
        // Few: each counts those above it, which takes no barrier but the last.
        int real = 0;
        for (int i0 = 0; i0 < n; i0 += (int)blockDim.x) {
            const int i = i0 + (int)threadIdx.x;
            const entry_t e = i < n ? list[i] : 0;
            if (e) {
                const int at = place_of(e, list, n);
                if (at < k) sorted[at] = e;
            }
            real += __syncthreads_count(e != 0);
        }
        *out = sorted;
        return min(real, k);
    }
    *out = sh->cand;
    // Far more candidates than places (a short row, all of it): bins over the range of a few more
    // than k of them, not over both signs.
    const entry_t floor = n > 2 * k + 64 ? select_threshold(list, n, k, k / 2 + 16, &sh->sel) : 1;
    return order_top(list, n, k, floor, sorted, sh->cand, &sh->sel);
}

// One row a block, or a cluster of blocks (CLUSTER) that take a slice of it each: few rows are
// spread over many SMs, and a slice's results meet in the first block's shared memory.  A row's
// slice is read once, a batch of each thread in flight while the one before is summed.
//
// Bound by the one read of the logits where no top is asked for: 4096 x 50257 bf16 with the entropy
// takes 67 us, 6.2 TB/s (some 40 instructions a vector of 8, over half of the issue slots).  With a top,
// the selection's instructions and its chain of barriers, a few us of a block's time, weigh as much as the
// reading of a row of some 10^4 logits: 2048 x 131072 with the top 64 takes 114 us (4.7 TB/s), 4096 x
// 32000 with the top 20 70 us.  One row is the length of that chain: 9.5 us with the top 20, 3.6 without.
template <typename T, bool ENT, bool TOP, bool CLUSTER>
__global__ void __launch_bounds__(kLpMaxThreads, 4) logprobs_kernel(const LpParams p) {
    using IO = Io<T>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __shared__ RowTotal sh_total[kLpMaxThreads / 32];
    __shared__ LpShare sh_share[CLUSTER ? kLpMaxCluster : 1];
    __shared__ int sh_above;
    const int tid = (int)threadIdx.x, nt = (int)blockDim.x;
    TopShared* sh = reinterpret_cast<TopShared*>(smem_raw);
    const int rank = CLUSTER ? (int)cluster_rank() : 0, blocks = CLUSTER ? (int)cluster_blocks() : 1;
    entry_t* sorted = reinterpret_cast<entry_t*>(smem_raw + sizeof(TopShared));
    entry_t* joined = sorted + max(kLpCand, blocks * p.top);  // in a cluster: all blocks' entries
    unsigned* segs = reinterpret_cast<unsigned*>(CLUSTER ? joined + blocks * p.top : joined);
    if constexpr (CLUSTER) cluster_arrive();  // "this block's shared memory exists"
    pdl_enter();
    const size_t row = blockIdx.x / (unsigned)blocks;
    const T* xr = static_cast<const T*>(p.x) + row * (size_t)p.ld;
    const RowCut<T, 32> cut(xr, p.V);
    const uint4* xv = reinterpret_cast<const uint4*>(xr + cut.head);
    const int per = ((cut.nvec + blocks - 1) / blocks + 1) & ~1;  // whole pairs
    const int lo = min(cut.nvec, rank * per), hi = min(cut.nvec, lo + per);
    const int step = kBatch * nt;
    uint4 u[kBatch];
    load_pairs<T>(u, xv, lo + 2 * tid, nt, hi);
    const int t = p.tokens ? p.tokens[row] : -1;
    const bool has = t >= 0 && t < p.V;
    const float nan = __int_as_float(0x7fc00000);
    const float xt = has ? IO::to_f(xr[t]) : nan;
    const float over = p.ranks ? xt : nan;  // values above it are counted
    if (tid == 0) sh_above = 0;
    RowSums<ENT> s;
    s.clear();
    const f2 c2 = f2_splat(p.c);
    int above = 0;
    float best = -INFINITY;
    const int seglen = (1 << p.seg_shift) / kBatch;
    int left = seglen, seg = tid;
    auto take = [&](const uint4 (&b)[kBatch], int v0) {
        const float m = s.template see_batch<T>(b, p.c);
        if (m > over) above += count_above<T>(b, over);
        if (m > -INFINITY) s.template add_batch<T>(b, c2);
        if constexpr (TOP) {
            if (p.seg_shift == 0) {  // a short row: this batch is the thread's only one
#pragma unroll
                for (int k = 0; k < kBatch; ++k, seg += nt) {
                    const float mk = vector_max<T>(b[k]);
                    segs[seg] = mk > -INFINITY ? order_key(mk) : 0;
                }
                return;
            }
            best = fmaxf(best, m);
            if (--left == 0) {
                segs[seg] = best > -INFINITY ? order_key(best) : 0;
                seg += nt;
                best = -INFINITY;
                left = seglen;
            }
        }
    };
    for (int v0 = lo + 2 * tid; v0 < hi; v0 += 2 * step) {
        uint4 ahead[kBatch];
        load_pairs<T>(ahead, xv, v0 + step, nt, hi);
        take(u, v0);
        if (v0 + step >= hi) break;
        load_pairs<T>(u, xv, v0 + 2 * step, nt, hi);
        take(ahead, v0 + step);
    }
    if constexpr (TOP) {
        for (; seg < p.nseg; seg += nt) {  // the last, unfilled segment, and those of no batch
            segs[seg] = best > -INFINITY ? order_key(best) : 0;
            best = -INFINITY;
        }
        if (tid < kLpLoose) segs[p.nseg + tid] = 0;
    }
    if (rank == 0 && tid < cut.nloose()) {
        const int col = cut.loose(tid);
        const float x = IO::to_f(xr[col]);
        s.add_one(x, p.c);
        above += x > over;
        if constexpr (TOP)
            if (x > -INFINITY) segs[p.nseg + tid] = order_key(x);
    }
    const RowTotal mine{s.ref, f2_lo(s.z2) + f2_hi(s.z2), ENT ? f2_lo(s.w2) + f2_hi(s.w2) : 0.f};
    __syncthreads();  // sh_above, segs
    above = __reduce_add_sync(kFullMask, above);
    if ((tid & 31) == 0 && above) atomicAdd(&sh_above, above);
    RowTotal a = block_total(mine, p.c, sh_total);
    __syncthreads();
    above = sh_above;
    const entry_t* list = nullptr;
    int n = 0;
    if constexpr (TOP) {
        n = collect_top<T>(p, xv, lo, hi, cut, sh, segs);
        list = sh->cand;
    }
    if constexpr (CLUSTER) {
        // Every block's sums and top entries go to the first, in the order of the blocks.
        cluster_wait();
        if (tid == 0) {
            const uint32_t to = in_block(&sh_share[rank], 0);
            st_cluster_f32(to, a.ref);
            st_cluster_f32(to + 4, a.z);
            st_cluster_f32(to + 8, a.w);
            st_cluster_f32(to + 12, __int_as_float(above));
        }
        if constexpr (TOP) {
            const uint32_t to = in_block(joined + rank * p.top, 0);
            entry_t* top;
            const int real = put_in_order(list, n, p.top, sorted, sh, &top);
            for (int i = tid; i < p.top; i += nt) st_cluster_u64(to + 8 * i, i < real ? top[i] : 0);
        }
        cluster_arrive();
        if (rank != 0) return;
        cluster_wait();
        a = sh_share[0].total;
        above = sh_share[0].above;
        for (int b = 1; b < blocks; ++b) {
            a = total_join(a, sh_share[b].total, p.c);
            above += sh_share[b].above;
        }
        if constexpr (TOP) {
            list = joined;
            n = blocks * p.top;
        }
    }
    const float r = a.ref == -INFINITY ? 0.f : a.ref;
    const float logz = logf(a.z);
    if (tid == 0) {
        if (p.lse) p.lse[row] = fmaf(r, p.scale, logz);
        if (ENT) p.entropy[row] = logz - kLn2 * a.w / a.z;
        // No token (t < 0): 0, of rank 0.  A token outside the row: NaN, of rank 0.
        if (p.logp) p.logp[row] = t < 0 ? 0.f : fmaf(xt - r, p.scale, -logz);
        if (p.ranks) p.ranks[row] = has ? above + 1 : 0;
    }
    if constexpr (TOP) {
        int* ids = p.top_ids + row * (size_t)p.top;
        float* lp = p.top_logp + row * (size_t)p.top;
        entry_t* top;
        const int real = put_in_order(list, n, p.top, sorted, sh, &top);
        for (int i = tid; i < p.top; i += nt) {
            const bool is = i < real;  // else: fewer logits above -inf than places
            ids[i] = is ? entry_col(top[i]) : -1;
            lp[i] = is ? fmaf(entry_value(top[i]) - r, p.scale, -logz) : -INFINITY;
        }
    }
}

template <typename T, bool CLUSTER>
const void* logprobs_variant(bool ent, bool top) {
    return top ? (ent ? (const void*)logprobs_kernel<T, true, true, CLUSTER>
                      : (const void*)logprobs_kernel<T, false, true, CLUSTER>)
               : (ent ? (const void*)logprobs_kernel<T, true, false, CLUSTER>
                      : (const void*)logprobs_kernel<T, false, false, CLUSTER>);
}

// Blocks a row is split over: as many as leave every SM no more than two blocks, of no less than 2048
// vectors each.  (One row of 131072 bf16 logits, top 20: 14.5 us in one block, 10.0 in 4, 9.6 in 8, 11.9
// in 16; of 16384 logits: 6.8 us in one block, 7.7 in 4.  64 rows of 131072: 18.2, 12.5 in 4, 16.0
// in 8; 200 rows: 25.4, 26.3 in 2.  Taken with 256 threads.)
int logprobs_cluster(int rows, int nvec, int sms) {
    int blocks = 1;
    while (blocks < kLpMaxCluster && (long long)rows * blocks * 2 <= 2 * sms && nvec / (blocks * 2) >= 2048)
        blocks *= 2;
    return blocks;
}

// Threads of a block at most, a power of two: 256, four blocks an SM.  Where there are rows for more than
// a wave of smaller blocks, 128: a row's fixed costs are by the warp (4096 x 50257 bf16: 68 us, 72 with
// 256; 4096 x 32000 with the top 20: 69 us, 80 with 256; but 700 x 50304: 28 us, 22 with 256; taken side by
// side, before the entropy's last step).
int logprobs_threads(int rows, int sms) { return rows > 8 * sms ? 128 : 256; }

template <typename T>
cudaError_t launch_logprobs_t(const LogprobsArgs& a, cudaStream_t stream) {
    constexpr int kVec = Io<T>::kVec;
    LpParams p;
    p.x = a.logits;
    p.ld = a.ld;
    p.tokens = a.tokens;
    p.V = a.V;
    p.top = a.top;
    p.scale = a.scale;
    p.c = a.scale * kLog2e;
    p.logp = a.logp;
    p.entropy = a.entropy;
    p.lse = a.lse;
    p.ranks = a.ranks;
    p.top_ids = a.top_ids;
    p.top_logp = a.top_logp;
    const int nvec = a.V / kVec;
    const int sms = device_info(-1).sms;
    const int blocks = logprobs_cluster(a.rows, nvec, sms);
    const int slice = ((nvec + blocks - 1) / blocks + 1) & ~1;
    const int most = logprobs_threads(a.rows, sms);
    // A batch for every thread, if there are that many.  The selection of a top is work for 4 warps
    // (1000 x 1024, top 20: 8.3 us), but for one where rows abound: more of them run at once (8192 x 1000,
    // top 20: 32 us, 39 with two warps, 54 with four).
    const int least = a.top > 0 && a.rows <= 8 * sms ? 7 : 5;  // log2
    int nt = 1 << least;
    p.nt_shift = least;
    while (nt < most && nt * kBatch < slice) {
        nt *= 2;
        ++p.nt_shift;
    }
    const int per = std::max(1, (slice + nt * kBatch - 1) / (nt * kBatch));  // batches of a thread
    int seglen = 1;
    p.seg_shift = 2;
    static_assert(kBatch == 1 << 2, "seg_shift counts vectors");
    // Segments enough that few of them hold a top element: what is read again is about top / segments of
    // the row, what the selection goes through is the segments.
    const int segments = std::min(std::max(32 * a.top, 512), kLpSegments);
    while (per * nt > seglen * segments) {
        seglen *= 2;
        ++p.seg_shift;
    }
    p.nseg = (per + seglen - 1) / seglen * nt;
    // Short rows have few batches: a segment for every vector, or all of the row would be candidates
    // (8192 x 256 with the top 10, four warps: 53 us, 63 with a segment for each batch; with one warp 27).
    if (per == 1) {
        p.seg_shift = 0;
        p.nseg = kBatch * nt;
    }
    const bool top = a.top > 0, ent = a.entropy != nullptr;
    size_t smem = 0;
    if (top) {
        const size_t joined = blocks > 1 ? (size_t)blocks * a.top : 0;
        smem = sizeof(TopShared) + (std::max((size_t)kLpCand, joined) + joined) * sizeof(entry_t) +
               ((size_t)p.nseg + kLpLoose) * sizeof(unsigned);
    }
    const void* kern = blocks > 1 ? logprobs_variant<T, true>(ent, top) : logprobs_variant<T, false>(ent, top);
    if (top) {
        const cudaError_t e = allow_smem(kern, smem);
        if (e != cudaSuccess) return e;
    }
    void* args[] = {&p};
    return launch_cluster(kern, dim3((unsigned)a.rows * (unsigned)blocks), dim3(nt), blocks, smem, stream, args);
}

// ---------------------------------------------------------------------------------------
// The gradient.  The forward left L and H, so every element stands for itself: one warp takes a
// piece of a row (some batches a lane), reads it, and writes the gradient of the same
// elements, which may be the logits' own place.  Bound by the read and the write: 4096 x 50257 bf16 with
// the entropy's part takes 126 us, 6.5 TB/s, 0.98 of what a copy gets.
//
// L in fp32 gives log q = z - L to half a step of L.  From kFineLse on (half a step is 2^-15 there) log Z
// gets lost in it -- altogether in a row masked throughout by its type's lowest value, where the
// softmax is uniform but z - L is 0 -- and the row's sums are formed again, about a value r of the row
// as in the forward: its first warp takes all of it, twice, and the others leave it (all rows so: 254 us,
// 2000 x 50304 fp32 209 us for 119, one row of 131072 bf16 105 us for 2).
// ---------------------------------------------------------------------------------------
constexpr int kLbThreads = 256;
constexpr int kLbBlocksPerSm = 4;
constexpr float kFineLse = 512.f;
// 0 * -inf is no term: log q is held where q is 0 in fp32 all the same, and no lower, or its product with a
// large upstream gradient would be infinite itself.
constexpr float kHeldLog = -128.f;

struct LbParams {
    const void* x;
    long long ld;
    const int* tokens;
    const float* lse;
    const float* entropy;
    const float* dlogp;
    const float* dent;
    long long pieces;  // rows * per_row
    int per_row;
    int V;
    float scale;
    void* dx;
    long long ldd;
};

// A warp's part of a row: vectors [lo, hi), and the loose elements where `loose`.
template <typename T>
struct LbPart {
    const T* xr;
    T* dr;
    RowCut<T> cut;
    int lo, hi;
    bool loose;
    __device__ __forceinline__ LbPart(const LbParams& p, size_t row, int part, int parts)
        : xr(static_cast<const T*>(p.x) + row * (size_t)p.ld),
          dr(static_cast<T*>(p.dx) + row * (size_t)p.ldd),
          cut(xr, p.V) {
        lo = (int)((long long)cut.nvec * part / parts);
        hi = (int)((long long)cut.nvec * (part + 1) / parts);
        loose = part == 0 && ((int)threadIdx.x & 31) < cut.nloose();
    }
    // A batch in flight while the one before is dealt with.
    template <typename F>
    __device__ __forceinline__ void each_batch(F deal) const {
        constexpr int kStep = 32 * kBatch;
        const uint4* xv = reinterpret_cast<const uint4*>(xr + cut.head);
        int v0 = lo + ((int)threadIdx.x & 31);
        if (v0 >= hi) return;
        uint4 u[kBatch], ahead[kBatch];
        load_batch<T>(u, xv, v0, 32, hi);
        while (true) {
            load_batch<T>(ahead, xv, v0 + kStep, 32, hi);
            deal(u, v0);
            if ((v0 += kStep) >= hi) break;
            load_batch<T>(u, xv, v0 + kStep, 32, hi);
            deal(ahead, v0);
            if ((v0 += kStep) >= hi) break;
        }
    }
};

// With lq = log q: dx = q (a + b lq), a = -scale (dlogp + dH entropy), b = -scale dH, and at the token sg =
// scale * dlogp more.
struct LbFactors {
    int t;
    float sg, b, a;
};

// The gradient of a part, lq = z - l, or (x - r) scale - l (ABOUT r).
template <typename T, bool ENT, bool WIDE, bool ABOUT>
__device__ __forceinline__ void put_gradient(const LbPart<T>& g, float scale, const LbFactors& k, float l, float r) {
    using IO = Io<T>;
    using PR = Pairs<T>;
    constexpr int kVec = IO::kVec;
    constexpr int H = PR::kPairs;
    const f2 s2 = f2_splat(scale), l2 = f2_splat(-l), e2 = f2_splat(kLog2e), a2 = f2_splat(k.a), b2 = f2_splat(k.b);
    g.each_batch([&](const uint4 (&u)[kBatch], int v0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int v = v0 + 32 * i;
            if (v >= g.hi) break;
            const int col = g.cut.col(v);
            f2 o[H];
            if constexpr (ABOUT)
                less<T>(u[i], r, o);
            else
                PR::unpack(u[i], o);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                f2 lq = f2_fma(o[h], s2, l2);
                const f2 y = f2_mul(lq, e2);
                const f2 q = f2_make(ex2_fast(f2_lo(y)), ex2_fast(f2_hi(y)));
                if constexpr (ENT) {
                    lq = f2_make(fmaxf(f2_lo(lq), kHeldLog), fmaxf(f2_hi(lq), kHeldLog));
                    o[h] = f2_mul(q, f2_fma(b2, lq, a2));
                } else {
                    o[h] = f2_mul(q, a2);
                }
            }
            const int in = k.t - col;  // the token's place in this vector
            if (in >= 0 && in < kVec) {
#pragma unroll
                for (int h = 0; h < H; ++h)
                    o[h] = f2_add(o[h], f2_make(in == 2 * h ? k.sg : 0.f, in == 2 * h + 1 ? k.sg : 0.f));
            }
            if constexpr (WIDE) {
                st_stream(g.dr + col, PR::pack(o));
            } else {
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    g.dr[col + 2 * h] = IO::from_f(f2_lo(o[h]));
                    g.dr[col + 2 * h + 1] = IO::from_f(f2_hi(o[h]));
                }
            }
        }
    });
    if (g.loose) {
        const int col = g.cut.loose((int)threadIdx.x & 31);
        const float x = IO::to_f(g.xr[col]);
        const float lq = fmaf(ABOUT ? x - r : x, scale, -l);
        const float q = ex2_fast(lq * kLog2e);
        const float o = ENT ? q * fmaf(k.b, fmaxf(lq, kHeldLog), k.a) : q * k.a;
        g.dr[col] = IO::from_f(col == k.t ? o + k.sg : o);
    }
}

// A whole row, from its own sums.
template <typename T, bool ENT, bool WIDE>
static __device__ __noinline__ void put_row_from_sums(const LbParams& p, size_t row, const LbFactors k) {
    const LbPart<T> g(p, row, 0, 1);
    const float c = p.scale * kLog2e;
    const f2 c2 = f2_splat(c);
    RowSums<false> s;
    s.clear();
    g.each_batch([&](const uint4 (&u)[kBatch], int) {
        if (s.see_batch<T>(u, c) > -INFINITY) s.add_batch<T>(u, c2);
    });
    if (g.loose) s.add_one(Io<T>::to_f(g.xr[g.cut.loose((int)threadIdx.x & 31)]), c);
    const RowTotal a = warp_total({s.ref, f2_lo(s.z2) + f2_hi(s.z2), 0.f}, c);
    put_gradient<T, ENT, WIDE, true>(g, p.scale, k, logf(a.z), a.ref == -INFINITY ? 0.f : a.ref);
}

// WIDE: logits and gradient lie at the same place of a 16-byte vector in every row.
template <typename T, bool ENT, bool WIDE>
__global__ void __launch_bounds__(kLbThreads, kLbBlocksPerSm)
    logprobs_bwd_kernel(const __grid_constant__ LbParams p) {
    using IO = Io<T>;
    pdl_enter();
    const int lane = (int)threadIdx.x & 31;
    const long long piece = (long long)blockIdx.x * (kLbThreads / 32) + (threadIdx.x >> 5);
    if (piece >= p.pieces) return;
    const size_t row = (size_t)(piece / p.per_row);
    const int part = (int)(piece % p.per_row);
    const LbPart<T> g(p, row, part, p.per_row);
    float dl = p.dlogp ? p.dlogp[row] : 0.f;
    const float de = ENT ? p.dent[row] : 0.f;
    const int t = p.dlogp ? p.tokens[row] : -1;
    const float lse = p.lse[row], hh = ENT ? p.entropy[row] : 0.f;
    if (t < 0) dl = 0.f;
    if (dl == 0.f && de == 0.f) {  // nothing flows back: 0, whatever the row holds
        if constexpr (WIDE) {
            for (int v = g.lo + lane; v < g.hi; v += 32) st_stream(g.dr + g.cut.col(v), make_uint4(0, 0, 0, 0));
        } else {
            for (int j = g.cut.col(g.lo) + lane; j < g.cut.col(g.hi); j += 32) g.dr[j] = IO::from_f(0.f);
        }
        if (g.loose) g.dr[g.cut.loose(lane)] = IO::from_f(0.f);
        return;
    }
    if (t >= p.V) dl = __int_as_float(0x7fc00000);
    const float sg = p.scale * dl, b = -p.scale * de;
    const LbFactors k{t, sg, b, ENT ? fmaf(b, hh, -sg) : -sg};
    if (fabsf(lse) >= kFineLse) {
        if (part == 0) put_row_from_sums<T, ENT, WIDE>(p, row, k);
        return;
    }
    put_gradient<T, ENT, WIDE, false>(g, p.scale, k, lse, 0.f);
}

template <typename T>
cudaError_t launch_logprobs_bwd_t(const LogprobsBwdArgs& a, cudaStream_t stream) {
    constexpr int kVec = Io<T>::kVec;
    LbParams p;
    p.x = a.logits;
    p.ld = a.ld;
    p.tokens = a.tokens;
    p.lse = a.lse;
    p.entropy = a.entropy;
    p.dlogp = a.dlogp;
    p.dent = a.dentropy;
    p.V = a.V;
    p.scale = a.scale;
    p.dx = a.dlogits;
    p.ldd = a.ldd;
    const int nvec = a.V / kVec;
    // Batches of a lane: one after another they hide a row's own loads (its log-sum, its token) and the
    // start of a warp, 151 us with one and 126 with four at 4096 x 50257 bf16 -- where there are some
    // waves of warps all the same (200 x 50257 fp32: 16.3 us with four, 15.0 with one).
    const long long resident = (long long)device_info(-1).sms * kLbBlocksPerSm * (kLbThreads / 32);
    int batches = 4;
    while (batches > 1 && (long long)a.rows * ((nvec + 31) / 32) < 3 * resident * kBatch * batches) batches /= 2;
    p.per_row = std::max(1, (nvec + 32 * kBatch * batches - 1) / (32 * kBatch * batches));
    p.pieces = (long long)a.rows * p.per_row;
    const bool wide = rows_congruent(a.logits, a.ld, a.dlogits, a.ldd, sizeof(T), a.rows);
    const bool ent = a.dentropy != nullptr;
    const void* kern = ent ? (wide ? (const void*)logprobs_bwd_kernel<T, true, true>
                                   : (const void*)logprobs_bwd_kernel<T, true, false>)
                           : (wide ? (const void*)logprobs_bwd_kernel<T, false, true>
                                   : (const void*)logprobs_bwd_kernel<T, false, false>);
    const long long blocks = (p.pieces + kLbThreads / 32 - 1) / (kLbThreads / 32);
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    void* args[] = {&p};
    return launch_kernel(kern, dim3((unsigned)blocks), dim3(kLbThreads), 0, stream, args, false);
}

}  // namespace

bool rows_congruent(const void* a, int64_t lda, const void* b, int64_t ldb, size_t esize, int rows) {
    const uint64_t base = reinterpret_cast<uintptr_t>(a) - reinterpret_cast<uintptr_t>(b);
    if (base & 15u) return false;
    return rows < 2 || (((uint64_t)lda - (uint64_t)ldb) * esize & 15u) == 0;
}

cudaError_t launch_logprobs(Dtype dt, const LogprobsArgs& a, cudaStream_t stream, int* launches) {
    cudaError_t e = dt == Dtype::F32 ? launch_logprobs_t<float>(a, stream)
                                     : launch_logprobs_t<__nv_bfloat16>(a, stream);
    *launches = e == cudaSuccess;
    return e;
}

cudaError_t launch_logprobs_bwd(Dtype dt, const LogprobsBwdArgs& a, cudaStream_t stream,
                                int* launches) {
    cudaError_t e = dt == Dtype::F32 ? launch_logprobs_bwd_t<float>(a, stream)
                                     : launch_logprobs_bwd_t<__nv_bfloat16>(a, stream);
    *launches = e == cudaSuccess;
    return e;
}

}  // namespace lnk
