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

// Copies of 16, 8 or 4 bytes into shared memory that go on by themselves: each thread commits its own in groups, and
// waits until all but its last N groups are there (for itself: others see them after a barrier).
template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_addr(to)), "l"(from), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Loads that stay where they are written, an iteration before their use.
__device__ __forceinline__ float load_ahead(const float* p) {
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t load_ahead(const uint8_t* p) {
    uint32_t v;
    asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
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

// The chunks that a lane has of a row: `at(k, c)` says whether it has a k-th and sets its address.  Those of a row that
// is not `inside` (the tensor's first and last) are left to end_chunks, which takes them one after another in one place
// of the code, and is called where they are needed: in line for each k they would take the registers, and merged with
// the loads they would make these wait where they are.
template <typename T, int NV, typename AT>
__device__ __forceinline__ void load_chunks(uint4 (&raw)[NV], bool inside, AT at) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const char* c;
        if (at(k, c) && inside) raw[k] = __ldcs(reinterpret_cast<const uint4*>(c));
    }
}

template <typename T, int NV, typename AT>
__device__ __forceinline__ void end_chunks(uint4 (&raw)[NV], bool inside, const Extent& t, AT at) {
    if (inside) return;
#pragma unroll 1
    for (int k = 0; k < NV; ++k) {
        const char* c;
        if (!at(k, c)) continue;
        const uint4 u = chunk_at<T>(c, t);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j == k) raw[j] = u;
    }
}

// A lane's vectors of a row: columns col(k) .. col(k) + V - 1 of its first n, col(k) a multiple of V, those behind n as
// anything; a vector without columns below n is left as it is.
template <typename T, int NV, typename COL>
__device__ __forceinline__ void load_vectors(uint4 (&raw)[NV], const RowIn<T>& r, int n, const Extent& t, COL col) {
    const unsigned s = (unsigned)reinterpret_cast<uintptr_t>(r.row) & 15u;  // the same in every lane
    const int sh = (int)s / (int)sizeof(T);
    auto one = [&](int k, const char*& c) {
        c = reinterpret_cast<const char*>(r.row + (col(k) - sh));
        return col(k) < n;
    };
    auto two = [&](int k, const char*& c) {
        c = reinterpret_cast<const char*>(r.row + (col(k) - sh + Io<T>::kVec));
        return s != 0 && col(k) - sh + Io<T>::kVec < n;
    };
    uint4 more[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) more[k] = make_uint4(0, 0, 0, 0);
    load_chunks<T>(raw, r.inside, one);
    load_chunks<T>(more, r.inside, two);
    end_chunks<T>(raw, r.inside, t, one);
    end_chunks<T>(more, r.inside, t, two);
    if (s == 0) return;
#pragma unroll
    for (int k = 0; k < NV; ++k) raw[k] = join_at(raw[k], more[k], s);
}

// One of them, col < n, a multiple of V.
template <typename T>
__device__ __forceinline__ uint4 load_columns(const RowIn<T>& r, int col, int n, const Extent& t) {
    uint4 u[1] = {make_uint4(0, 0, 0, 0)};
    load_vectors<T>(u, r, n, t, [&](int) { return col; });
    return u[0];
}

// Elements from .. to - 1 of lane `src`'s vector, each stored by a lane of its own: element e to p + e (p, src, from
// and to the same in a group of L lanes; all lanes of the warp call it).
template <typename T, int L>
__device__ __forceinline__ void store_some(T* p, const uint4& u, int src, int from, int to) {
    const uint32_t x = __shfl_sync(kFullMask, u.x, src, L), y = __shfl_sync(kFullMask, u.y, src, L);
    const uint32_t z = __shfl_sync(kFullMask, u.z, src, L), w = __shfl_sync(kFullMask, u.w, src, L);
    const int e = threadIdx.x & (L - 1), i = sizeof(T) == 2 ? e >> 1 : e;
    const uint32_t v = i & 2 ? (i & 1 ? w : z) : (i & 1 ? y : x);
    if (e >= from && e < to && e < Io<T>::kVec) {
        if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint16_t*>(p + e) = (uint16_t)(v >> (16 * (e & 1)));
        else
            *reinterpret_cast<uint32_t*>(p + e) = v;
    }
}

// Groups of L lanes store L chunks of a row that starts `sh` elements into the chunk of place 0 and has its end at
// place `end`: lane l's, at p, at places from + l V .. from + l V + V - 1, whole, or those of its elements that are the
// row's.  Called by all lanes of the warp, with one `from`.
template <typename T, int L>
__device__ __forceinline__ void store_chunks(T* p, int from, int sh, int end, const uint4& u) {
    constexpr int V = Io<T>::kVec;
    const int lane = threadIdx.x & (L - 1), col = from + lane * V;
    if (col >= sh && col + V <= end) __stcs(reinterpret_cast<uint4*>(p), u);
    if (from == 0 && (L == 32 ? sh > 0 : __any_sync(kFullMask, sh > 0)))
        store_some<T, L>(p - lane * V, u, 0, sh, sh > 0 ? end : 0);
    const int left = end - from, last = left / V;  // the chunk with the row's end inside, if it is one of these
    const bool part = left > 0 && left < L * V && left % V != 0 && !(from == 0 && last == 0 && sh > 0);
    if (L == 32 ? part : __any_sync(kFullMask, part))
        store_some<T, L>(p + (last - lane) * V, u, last, 0, part ? left - last * V : 0);
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
        const int lane = threadIdx.x & (L - 1), base = col - lane * V;
        if (L == 32 ? s == 0 : __all_sync(kFullMask, s == 0)) {
            if (col + V <= n) __stcs(reinterpret_cast<uint4*>(p), u);
            const int end = n <= base ? 0 : (n - base) / V;  // the vector that the row ends in
            if (L == 32 ? n % V != 0 : __any_sync(kFullMask, n % V != 0))
                store_some<T, L>(row + (base + end * V), u, end, 0, n <= base || end >= L ? 0 : n - base - end * V);
            return;
        }
        const int over = (int)s / (int)sizeof(T);  // elements of mine that belong to the next lane's chunk
        uint4 before;
        before.x = __shfl_sync(kFullMask, u.x, lane + L - 1, L);
        before.y = __shfl_sync(kFullMask, u.y, lane + L - 1, L);
        before.z = __shfl_sync(kFullMask, u.z, lane + L - 1, L);
        before.w = __shfl_sync(kFullMask, u.w, lane + L - 1, L);
        const uint4 next = before;  // (lane 0: the piece's last vector)
        if (lane == 0 && !first) before = carry;
        carry = next;
        // The chunk of the `over` elements before mine and my first V - over; the first lane of all has the latter alone.
        const uint4 c = s == 0 ? u : join_at(before, u, 16 - s);
        const int at = col - over;
        if (at + V <= n && (lane > 0 || !first || s == 0)) *reinterpret_cast<uint4*>(p - over) = c;
        if (first) store_some<T, L>(row + base, u, 0, 0, s == 0 ? 0 : min(V - over, n - base));
        // The chunk that the row ends in, and the last piece's last `over` elements.
        const int end = n <= base - over ? L : (n - (base - over)) / V;
        const bool inner = end < L && !(end == 0 && first && s != 0) && n > base - over + end * V;
        if (L == 32 ? inner : __any_sync(kFullMask, inner))
            store_some<T, L>(row + (base - over + end * V), c, min(end, L - 1), 0, inner ? n - (base - over + end * V) : 0);
        const bool outer = s != 0 && (last || base + L * V >= n);
        if (L == 32 ? outer : __any_sync(kFullMask, outer))
            store_some<T, L>(row + (base + (L - 1) * V), u, L - 1, V - over, outer ? n - (base + (L - 1) * V) : 0);
    }
};

}  // namespace
}  // namespace lnk
