// top_select.cuh -- the largest k of a row of logits, by a block: order keys and the selection
// of a threshold by histograms of a shrinking range.
//
// An entry is one 64-bit word: the value as an unsigned integer of the same order above the
// complement of its column, so that entries of a row are all different, larger means "larger
// value, or the same value in a lower column", and 0 is no entry (-inf and NaN give none).
#pragma once

#include "ln_device.cuh"

namespace lnk {

using entry_t = unsigned long long;

// x > -inf, not NaN.  -0 counts as +0.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t b = __float_as_uint(__fadd_rn(x, 0.f));
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ entry_t make_entry(float x, int col) {
    return ((entry_t)order_key(x) << 32) | (uint32_t)~(uint32_t)col;
}
__device__ __forceinline__ float entry_value(entry_t e) { return order_value((uint32_t)(e >> 32)); }
__device__ __forceinline__ int entry_col(entry_t e) { return (int)~(uint32_t)e; }

constexpr int kSelBins = 256;
constexpr int kSelBinBits = 8;

struct __align__(16) SelectShared {
    unsigned bins[kSelBins];
    unsigned cursor[kSelBins];
    int base[kSelBins];
    entry_t lo, hi;
    unsigned least, most;
    int above, taken, done;
};

// A threshold t with at least k, and where the values allow it at most k + slack, of the n entries (or
// bare keys, E = unsigned) >= t; the list may hold zeros (no entry), which never count.  With
// k + slack entries or fewer: 1 (every entry).
//
// One step spreads the entries of a range [lo, hi] over at most 256 bins of equal width (a power
// of two), finds from the top the bin that holds the k-th, and goes on within it.  The first range
// is that of the entries themselves, so that logits of any size fill the bins; with some slack one
// step is usually enough.  Every thread of the block calls it, with the entries in shared memory
// and visible; it returns the same value to all.
template <typename E>
static __device__ __noinline__ E select_threshold(const E* list, int n, int k, int slack, SelectShared* sh) {
    constexpr int kBits = 8 * sizeof(E), kKeyShift = kBits - 32;
    const int tid = (int)threadIdx.x, nt = (int)blockDim.x, lane = tid & 31;
    unsigned mn = ~0u, mx = 0;
    int have = 0;
#pragma unroll 1
    for (int i = tid; i < n; i += nt) {
        const E e = list[i];
        if (e == 0) continue;
        const unsigned key = (unsigned)(e >> kKeyShift);
        mn = min(mn, key);
        mx = max(mx, key);
        ++have;
    }
    if (tid == 0) {
        sh->above = sh->taken = sh->done = 0;
        sh->least = ~0u;
        sh->most = 0;
    }
    __syncthreads();
    mn = __reduce_min_sync(kFullMask, mn);
    mx = __reduce_max_sync(kFullMask, mx);
    have = __reduce_add_sync(kFullMask, have);
    if (lane == 0 && have) {
        atomicMin(&sh->least, mn);
        atomicMax(&sh->most, mx);
        atomicAdd(&sh->taken, have);
    }
#pragma unroll 1
    for (int i = tid; i < kSelBins; i += nt) sh->bins[i] = 0;
    __syncthreads();
    if (sh->taken <= k + slack) {
        __syncthreads();
        return 1;
    }
    E lo = (E)sh->least << kKeyShift, hi = (E)(((E)sh->most << kKeyShift) | (((E)1 << kKeyShift) - 1));
    // Each step leaves a range of at most 2^-7 of the one before.
#pragma unroll 1
    for (int step = 0; step < 10; ++step) {
        const int width = sizeof(E) == 8 ? 64 - __clzll((long long)(hi - lo)) : 32 - __clz((int)(hi - lo));
        const int shift = max(0, width - kSelBinBits);
#pragma unroll 1
        for (int i = tid; i < n; i += nt) {
            const E e = list[i];
            if (e >= lo && e <= hi) atomicAdd(&sh->bins[(int)((e - lo) >> shift)], 1u);
        }
        __syncthreads();
        if (tid < 32) {
            // Lane l's share, from the top: bins 255 - 8 l down to 248 - 8 l.
            const int need = k - sh->above;
            const uint4 p = *reinterpret_cast<const uint4*>(&sh->bins[kSelBins - 8 - 8 * lane]);
            const uint4 q = *reinterpret_cast<const uint4*>(&sh->bins[kSelBins - 4 - 8 * lane]);
            const int mine = (int)(p.x + p.y + p.z + p.w + q.x + q.y + q.z + q.w);
            int upto = mine;  // the sum of lanes 0 .. lane
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFullMask, upto, o);
                if (lane >= o) upto += v;
            }
            const int who = __ffs(__ballot_sync(kFullMask, upto >= need)) - 1;  // never none: n > k
            if (lane == who) {
                const unsigned c[8] = {q.w, q.z, q.y, q.x, p.w, p.z, p.y, p.x};  // from the top
                int cum = upto - mine, bin = kSelBins - 1 - 8 * lane, here = 0;
                bool found = false;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (found) continue;
                    here = (int)c[i];
                    cum += here;
                    if (cum >= need)
                        found = true;
                    else
                        --bin;
                }
                const E nlo = lo + ((E)bin << shift);
                sh->done = shift == 0 || sh->above + cum <= k + slack;
                sh->above += cum - here;
                sh->lo = nlo;
                sh->hi = nlo + min((E)(hi - nlo), (E)(((E)1 << shift) - 1));  // (the bin may end past the type's range)
            }
        }
        __syncthreads();
        lo = (E)sh->lo;
        hi = (E)sh->hi;
        if (sh->done) break;
#pragma unroll 1
        for (int i = tid; i < kSelBins; i += nt) sh->bins[i] = 0;
        __syncthreads();
    }
    __syncthreads();  // *sh is free for the next use
    return lo;
}

// Each entry's place among n entries in falling order, by counting the larger ones.
__device__ __forceinline__ int place_of(entry_t e, const entry_t* list, int n) {
    int r = 0;
#pragma unroll 8
    for (int i = 0; i < n; ++i) r += list[i] > e;
    return r;
}

// The k largest, or all, of the entries >= floor among n, in falling order, into `out`; returns how many
// there are.  `list`, `sorted` (for n entries) and `out` (for k, not `sorted`, perhaps `list`) are in
// shared memory.  Zeros are no entries.
//
// A counting sort by the leading bits of the value, spread over the values' own range: entries go to
// their bin's place in `sorted`, and only entries of the same bin are compared with one another.
// (Comparing every entry with every other takes 5 us for 512 of them.)
static __device__ __noinline__ int order_top(const entry_t* list, int n, int k, entry_t floor,
                                             entry_t* sorted, entry_t* out, SelectShared* sh) {
    const int tid = (int)threadIdx.x, nt = (int)blockDim.x, lane = tid & 31;
    if (tid == 0) {
        sh->least = ~0u;
        sh->most = 0;
    }
#pragma unroll 1
    for (int i = tid; i < kSelBins; i += nt) sh->bins[i] = sh->cursor[i] = 0;
    floor = max(floor, (entry_t)1);
    unsigned mn = ~0u, mx = 0;
#pragma unroll 1
    for (int i = tid; i < n; i += nt) {
        const entry_t e = list[i];
        if (e < floor) continue;
        mn = min(mn, (unsigned)(e >> 32));
        mx = max(mx, (unsigned)(e >> 32));
    }
    __syncthreads();
    mn = __reduce_min_sync(kFullMask, mn);
    mx = __reduce_max_sync(kFullMask, mx);
    if (lane == 0 && mx) {
        atomicMin(&sh->least, mn);
        atomicMax(&sh->most, mx);
    }
    __syncthreads();
    const unsigned least = sh->least;
    const int shift = max(0, 32 - __clz((int)(sh->most - least)) - kSelBinBits);
#pragma unroll 1
    for (int i = tid; i < n; i += nt) {
        const entry_t e = list[i];
        if (e >= floor) atomicAdd(&sh->bins[((unsigned)(e >> 32) - least) >> shift], 1u);
    }
    __syncthreads();
    if (tid < 32) {
        // base[b]: the entries in bins above b.  Lane l has bins 255 - 8 l down to 248 - 8 l.
        int mine = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) mine += (int)sh->bins[kSelBins - 1 - 8 * lane - i];
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFullMask, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) sh->taken = upto;
        upto -= mine;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sh->base[kSelBins - 1 - 8 * lane - i] = upto;
            upto += (int)sh->bins[kSelBins - 1 - 8 * lane - i];
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < n; i += nt) {
        const entry_t e = list[i];
        if (e < floor) continue;
        const unsigned b = ((unsigned)(e >> 32) - least) >> shift;
        if (sh->base[b] < k) sorted[sh->base[b] + (int)atomicAdd(&sh->cursor[b], 1u)] = e;
    }
    __syncthreads();
    const int have = sh->taken;
#pragma unroll 1
    for (int i = tid; i < have; i += nt) {
        // What stands at i belongs to a bin that has been filled, or nothing has.
        const entry_t e = sorted[i];
        const unsigned b = ((unsigned)(e >> 32) - least) >> shift;
        if (b >= kSelBins || sh->base[b] >= k) continue;
        const int from = sh->base[b], end = from + (int)sh->bins[b];
        if (i < from || i >= end) continue;
        int at = from;
#pragma unroll 1
        for (int j = from; j < end; ++j) at += sorted[j] > e;
        if (at < k) out[at] = e;
    }
    __syncthreads();
    return min(have, k);
}

}  // namespace lnk
