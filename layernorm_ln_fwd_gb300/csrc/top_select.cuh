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

constexpr int kSelBins = 1024;
constexpr int kSelBinBits = 10;

struct SelectShared {
    unsigned bins[kSelBins];
    entry_t lo, hi;
    entry_t wmin[32], wmax[32];
    int above, taken, done;
};

// A threshold t with at least k, and at most k + slack, of the n entries >= t; n may hold zeros
// (no entry), which never count.  With fewer than k entries: 1 (every entry).  Entries are
// different from one another, except that slack 0 needs it: then exactly k are >= t.
//
// One step spreads the entries of a range [lo, hi] over at most 1024 bins of equal width (a power
// of two), finds from the top the bin that holds the k-th, and goes on within it.  The first
// range is that of the entries themselves, so that logits of any size fill the bins; a step takes
// 10 bits off the range, two or three steps in all.  Every thread of the block calls it, with
// the entries in shared memory and visible; it returns the same value to all.
__device__ __forceinline__ entry_t select_threshold(const entry_t* list, int n, int k, int slack,
                                                    SelectShared* sh) {
    const int tid = (int)threadIdx.x, nt = (int)blockDim.x, lane = tid & 31, warp = tid >> 5;
    entry_t mn = ~0ull, mx = 0;
    int have = 0;
    for (int i = tid; i < n; i += nt) {
        const entry_t e = list[i];
        if (e) {
            mn = min(mn, e);
            mx = max(mx, e);
            ++have;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        mn = min(mn, __shfl_xor_sync(kFullMask, mn, o));
        mx = max(mx, __shfl_xor_sync(kFullMask, mx, o));
    }
    have = __reduce_add_sync(kFullMask, have);
    if (tid == 0) {
        sh->above = 0;
        sh->taken = 0;
        sh->done = 0;
        sh->lo = ~0ull;
        sh->hi = 0;
    }
    __syncthreads();
    if (lane == 0) {
        sh->wmin[warp] = mn;
        sh->wmax[warp] = mx;
        atomicAdd(&sh->taken, have);
    }
    __syncthreads();
    if (sh->taken <= k + slack) {
        __syncthreads();
        return 1;
    }
    if (warp == 0) {
        const int nw = nt >> 5;
        mn = lane < nw ? sh->wmin[lane] : ~0ull;
        mx = lane < nw ? sh->wmax[lane] : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            mn = min(mn, __shfl_xor_sync(kFullMask, mn, o));
            mx = max(mx, __shfl_xor_sync(kFullMask, mx, o));
        }
        if (lane == 0) {
            sh->lo = mn;
            sh->hi = mx;
        }
    }
    // At most 7 steps: each leaves a range of at most 2^-9 of the one before.
    for (int step = 0; step < 8; ++step) {
        for (int i = tid; i < kSelBins; i += nt) sh->bins[i] = 0;
        __syncthreads();
        const entry_t lo = sh->lo, hi = sh->hi;
        const int shift = max(0, 64 - __clzll((long long)(hi - lo)) - kSelBinBits);
        for (int i = tid; i < n; i += nt) {
            const entry_t e = list[i];
            if (e >= lo && e <= hi) atomicAdd(&sh->bins[(int)((e - lo) >> shift)], 1u);
        }
        __syncthreads();
        if (warp == 0) {
            // Lane l's share, from the top: bins 1023 - 32 l down to 992 - 32 l (read in an order
            // that keeps the lanes on different banks).
            const int need = k - sh->above;
            int mine = 0;
#pragma unroll 8
            for (int i = 0; i < 32; ++i) mine += (int)sh->bins[kSelBins - 1 - 32 * lane - ((i + lane) & 31)];
            int upto = mine;  // the sum of lanes 0 .. lane
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFullMask, upto, o);
                if (lane >= o) upto += v;
            }
            const int who = __ffs(__ballot_sync(kFullMask, upto >= need)) - 1;  // never none: n > k
            const int before = __shfl_sync(kFullMask, upto - mine, who);
            const int bin = kSelBins - 1 - 32 * who - lane;
            const int here = (int)sh->bins[bin];
            int within = here;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFullMask, within, o);
                if (lane >= o) within += v;
            }
            const unsigned hit = __ballot_sync(kFullMask, before + within >= need);
            if (lane == __ffs(hit) - 1) {
                const int cum = before + within;  // entries of the range in this bin and above
                const entry_t nlo = lo + ((entry_t)bin << shift);
                sh->done = shift == 0 || sh->above + cum <= k + slack;
                sh->above += cum - here;
                sh->lo = nlo;
                sh->hi = min(hi, nlo + (((entry_t)1 << shift) - 1));
            }
        }
        __syncthreads();
        if (sh->done) break;
    }
    const entry_t t = sh->lo;
    __syncthreads();  // *sh is free for the next use
    return t;
}

// Each entry's place among n entries in falling order, by counting the larger ones: for n up to a
// few hundred, one pass over shared memory that every lane reads at the same address.
__device__ __forceinline__ int place_of(entry_t e, const entry_t* list, int n) {
    int r = 0;
    for (int i = 0; i < n; ++i) r += list[i] > e;
    return r;
}

}  // namespace lnk
