// row_io.cuh -- 16-byte vectors of rows that start at any element: shared by the softmax with a
// relative position bias and the 8-bit checkpoints.
//
// A thread holds the V = 16 / sizeof(T) columns from a multiple of V of its row.  Where the row starts
// on a 16-byte boundary that is one 128-bit access.  Elsewhere (an odd number of columns, a view) every
// row starts s bytes behind a boundary: a load takes the two aligned chunks that its vector lies in (the
// second is its neighbour's first, so that it comes from L1) and moves them together; a store takes the
// last s bytes of the lane before it and writes the one aligned chunk that the two share.  Either costs
// some fifteen integer instructions a vector, against V accesses of one element each with 16 bytes
// between lanes, which fill one 32-byte sector of each 16 that they touch.
#pragma once

#include "ln_device.cuh"

namespace lnk {
namespace {

// The elements of a tensor: from lo, up to hi.  Aligned chunks are read whole only inside it.
struct Extent {
    const char* lo;
    const char* hi;
};

// The 16 bytes that start s bytes into the 32 bytes (a, b), 0 < s < 16, s a multiple of 2.
__device__ __forceinline__ uint4 join_at(const uint4& a, const uint4& b, unsigned s) {
    uint32_t w[6];
    const bool two = s & 8u, one = s & 4u;
    w[0] = two ? a.z : a.x;
    w[1] = two ? a.w : a.y;
    w[2] = two ? b.x : a.z;
    w[3] = two ? b.y : a.w;
    w[4] = two ? b.z : b.x;
    w[5] = two ? b.w : b.y;
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = one ? w[i + 1] : w[i];
    const unsigned bits = (s & 2u) * 8u;
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

__device__ __forceinline__ void set_word(uint4& u, int i, uint32_t v) {
    if (i == 0) u.x = v;
    if (i == 1) u.y = v;
    if (i == 2) u.z = v;
    if (i == 3) u.w = v;
}

// The first `count` elements of a vector, zeros behind them.
template <typename T>
__device__ __forceinline__ uint4 first_of(const uint4& u, int count) {
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2)
            w[i] &= (2 * i < count ? 0xffffu : 0u) | (2 * i + 1 < count ? 0xffff0000u : 0u);
        else
            w[i] = i < count ? w[i] : 0u;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A vector without its first `count` elements: zeros in their place.
template <typename T>
__device__ __forceinline__ uint4 behind(const uint4& u, int count) {
    const uint4 f = first_of<T>(u, count);
    return make_uint4(u.x ^ f.x, u.y ^ f.y, u.z ^ f.z, u.w ^ f.w);
}

// The aligned chunk at c, of which at least one element is the tensor's; at the tensor's ends the
// elements inside it alone, zeros elsewhere.
template <typename T>
__device__ __forceinline__ uint4 chunk_at(const char* c, const Extent& t) {
    if (c >= t.lo && c + 16 <= t.hi) return *reinterpret_cast<const uint4*>(c);
    uint4 u = make_uint4(0, 0, 0, 0);
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
        const char* q = c + 4 * i;
        uint32_t w = 0;
        if constexpr (sizeof(T) == 2) {
            if (q >= t.lo && q < t.hi) w = *reinterpret_cast<const uint16_t*>(q);
            if (q + 2 >= t.lo && q + 2 < t.hi) w |= (uint32_t)*reinterpret_cast<const uint16_t*>(q + 2) << 16;
        } else {
            if (q >= t.lo && q < t.hi) w = *reinterpret_cast<const uint32_t*>(q);
        }
        set_word(u, i, w);
    }
    return u;
}

// A row to read: whether the chunks at its ends are the tensor's as well.
template <typename T>
struct RowIn {
    const T* row;
    bool inside;
    __device__ __forceinline__ RowIn(const T* r, int n, const Extent& t)
        : row(r),
          inside(reinterpret_cast<const char*>(r) - 15 >= t.lo && reinterpret_cast<const char*>(r + n) + 15 <= t.hi) {}
};

// The vector of load_columns in a tensor's first or last row (a call: rare, and too large to have in line).
template <typename T>
__device__ __noinline__ uint4 load_at_end(const char* p, bool two, Extent t) {
    const unsigned s = (unsigned)reinterpret_cast<uintptr_t>(p) & 15u;
    const uint4 a = chunk_at<T>(p - s, t);
    return s == 0 ? a : join_at(a, two ? chunk_at<T>(p - s + 16, t) : make_uint4(0, 0, 0, 0), s);
}

// Columns col .. col + V - 1 of a row whose first n > col columns are wanted; those behind them come
// as anything.
template <typename T>
__device__ __forceinline__ uint4 load_columns(const RowIn<T>& r, int col, int n, const Extent& t) {
    constexpr int V = Io<T>::kVec;
    const char* p = reinterpret_cast<const char*>(r.row + col);
    const unsigned s = (unsigned)reinterpret_cast<uintptr_t>(p) & 15u;  // the same in every lane
    const bool two = s != 0 && col + (16 - (int)s) / (int)sizeof(T) < n;  // the second chunk has columns
    if (!r.inside && (s != 0 || col + V > n)) return load_at_end<T>(p, two, t);
    const uint4 a = *reinterpret_cast<const uint4*>(p - s);
    if (s == 0) return a;
    return join_at(a, two ? *reinterpret_cast<const uint4*>(p - s + 16) : make_uint4(0, 0, 0, 0), s);
}

// The aligned chunk that begins at column col of a row (col may lie before it): the row's elements, others'
// around them.
template <typename T>
__device__ __forceinline__ uint4 load_chunk(const RowIn<T>& r, int col, const Extent& t) {
    const char* p = reinterpret_cast<const char*>(r.row + col);
    return r.inside ? __ldcs(reinterpret_cast<const uint4*>(p)) : load_at_end<T>(p, false, t);
}

// One element of a vector, as it is stored.
template <typename T>
__device__ __forceinline__ void store_element(T* p, const uint4& u, int e) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint16_t*>(p) = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    else
        *reinterpret_cast<uint32_t*>(p) = w[e];
}

// Places col .. col + V - 1 of a row that starts `sh` elements into the chunk of place 0 and has its end at
// place `end`: the chunk whole, or those of its elements that are the row's.
template <typename T>
__device__ __forceinline__ void store_chunk(T* row, int col, int sh, int end, const uint4& u) {
    constexpr int V = Io<T>::kVec;
    T* p = row + (col - sh);
    if (col >= sh && col + V <= end) {
        __stcs(reinterpret_cast<uint4*>(p), u);
    } else if (col < end) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (col + e >= sh && col + e < end) store_element(p + e, u, e);
    }
}

// A row's (or a part's) vectors on their way out, by groups of L lanes: pieces of L vectors that follow one another,
// lane l's of a piece with columns col .. col + V - 1, col = the piece's first + l V, of a row of n columns (those of n
// and more are not stored; rows may differ from group to group).  `first` and `last`: the first and the last piece,
// whose outer ends lie in chunks shared with others (a piece that ends at n or behind may be the last unsaid).
// Called by all lanes of the warp.
template <typename T, int L>
struct RowOut {
    uint4 carry;  // lane 0: the vector before the piece

    __device__ __forceinline__ void put(T* row, int col, int n, const uint4& u, bool first, bool last) {
        constexpr int V = Io<T>::kVec;
        T* p = row + col;
        const unsigned s = (unsigned)reinterpret_cast<uintptr_t>(p) & 15u;  // the same in every lane of a group
        if (L == 32 ? s == 0 : __all_sync(kFullMask, s == 0)) {
            if (col + V <= n) {
                __stcs(reinterpret_cast<uint4*>(p), u);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (col + e < n) store_element(p + e, u, e);
            }
            return;
        }
        const int lane = threadIdx.x & (L - 1);
        const int over = (int)s / (int)sizeof(T);  // elements of mine that belong to the next lane's chunk
        uint4 before;
        before.x = __shfl_sync(kFullMask, u.x, lane + L - 1, L);
        before.y = __shfl_sync(kFullMask, u.y, lane + L - 1, L);
        before.z = __shfl_sync(kFullMask, u.z, lane + L - 1, L);
        before.w = __shfl_sync(kFullMask, u.w, lane + L - 1, L);
        const uint4 next = before;  // (lane 0: the piece's last vector)
        if (lane == 0 && !first) before = carry;
        carry = next;
        if (lane > 0 || !first || s == 0) {  // the chunk of the `over` elements before mine and my first V - over
            const uint4 c = s == 0 ? u : join_at(before, u, 16 - s);
            if (col - over + V <= n) {
                *reinterpret_cast<uint4*>(p - over) = c;
            } else if (col - over < n) {
                put_some(p - over, c, 0, n - (col - over));
            }
        } else {
            put_some(p, u, 0, min(V - over, n - col));
        }
        // The last piece's last `over` elements (where the row ends with the piece before, no lane takes them either).
        if (lane == L - 1 && s != 0 && (last || col + V >= n)) put_some(p, u, V - over, n - col);
    }

    // Elements from .. to - 1 of a vector.
    static __device__ __forceinline__ void put_some(T* p, const uint4& u, int from, int to) {
#pragma unroll
        for (int e = 0; e < Io<T>::kVec; ++e)
            if (e >= from && e < to) store_element(p + e, u, e);
    }
};

}  // namespace
}  // namespace lnk
