// vocab.cuh -- device-side building blocks of the operators over rows of logits
// (logprobs.cu, distill.cu): a row as 16-byte vectors and loose ends, and the running
// softmax sums of a row.
#pragma once

#include <math.h>

#include "ln_device.cuh"

namespace lnk {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// A row of V logits at any element-aligned address: `head` loose elements up to the first
// 16-byte boundary, `nvec` aligned vectors, `tail` loose elements behind them.  Rows of an odd
// length one after another start at a different place of a vector each; cutting every row at its
// own boundaries keeps all but at most 2 * (kVec - 1) elements on 16-byte accesses.
template <typename T>
struct RowCut {
    int head, nvec, tail;
    __device__ __forceinline__ RowCut(const T* row, int V) {
        constexpr int kVec = Io<T>::kVec;
        const int mis = (int)(reinterpret_cast<uintptr_t>(row) & 15u) / (int)sizeof(T);
        head = min(V, (kVec - mis) % kVec);
        nvec = (V - head) / kVec;
        tail = V - head - nvec * kVec;
    }
    // The column of loose element i, 0 <= i < head + tail.
    __device__ __forceinline__ int loose(int i) const {
        return i < head ? i : nvec * Io<T>::kVec + i;
    }
    __device__ __forceinline__ int nloose() const { return head + tail; }
    // The first column of vector v.
    __device__ __forceinline__ int col(int v) const { return head + v * Io<T>::kVec; }
};

// The largest value of a vector in fp32 (exact).  NaN loses against a number.
template <typename T>
__device__ __forceinline__ float vector_max(const uint4& u) {
    if constexpr (sizeof(T) == 2) {
        __nv_bfloat162 a, b, c, d;
        memcpy(&a, &u.x, 4);
        memcpy(&b, &u.y, 4);
        memcpy(&c, &u.z, 4);
        memcpy(&d, &u.w, 4);
        const __nv_bfloat162 m = __hmax2(__hmax2(a, b), __hmax2(c, d));
        return fmaxf(__low2float(m), __high2float(m));
    } else {
        return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)),
                     fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
    }
}

// Running sums of a softmax over the values seen so far, about a reference value `ref`:
//   u = (x - ref) * c,  z = sum 2^u,  w = sum 2^u u          (c = scale * log2 e).
// The reference is a value of the row and at most 2^kSlack below the largest one in weight: it is
// replaced, and the sums rescaled, only when a value exceeds it by more than that.  A plain running
// maximum moves for some lane of a warp in almost every step of a row of a few thousand values;
// this one moves once or twice a row, the sums lose nothing (they are only scaled by a power of
// two's neighbourhood), and log z - ln 2 w / z has terms of at most kSlack to cancel.
// ref = -inf: no value above -inf yet; u is then taken about 0, so that -inf adds nothing and a
// NaN still reaches z.  The differences x - ref are taken before the product with c: a value next
// to the reference keeps its exact distance whatever the size of both.
constexpr float kSlack = 8.f;

template <bool ENT>
struct RowSums {
    float ref, refu;  // refu: ref, or 0 while ref is -inf
    f2 z2, w2;
    __device__ __forceinline__ void clear() {
        ref = -INFINITY;
        refu = 0.f;
        z2 = f2_splat(0.f);
        w2 = f2_splat(0.f);
    }
    // Move the reference to m > ref.
    __device__ __forceinline__ void rebase(float m, float c) {
        if (ref != -INFINITY) {
            const float d = (ref - m) * c;
            const f2 f = f2_splat(ex2_fast(d));
            if constexpr (ENT) w2 = f2_mul(f, f2_fma(z2, f2_splat(fmaxf(d, -1e30f)), w2));
            z2 = f2_mul(f, z2);
        }
        ref = refu = m;
    }
    __device__ __forceinline__ void see(float m, float c) {
        if (m > ref && !((m - ref) * c <= kSlack)) rebase(m, c);
    }
    // Add the pairs of one vector whose largest value see() has been given.
    template <int H>
    __device__ __forceinline__ void add(const f2 (&x)[H], f2 c2) {
        const f2 r2 = f2_splat(-refu);
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const f2 u = f2_mul(f2_add(x[h], r2), c2);
            const f2 e = f2_make(ex2_fast(f2_lo(u)), ex2_fast(f2_hi(u)));
            z2 = f2_add(z2, e);
            // 0 * -inf is no term: the exponent is held at a value whose weight is 0 as well.
            if constexpr (ENT) w2 = f2_fma(e, f2_make(fmaxf(f2_lo(u), -1e30f), fmaxf(f2_hi(u), -1e30f)), w2);
        }
    }
    __device__ __forceinline__ void add_one(float x, float c) {
        see(x, c);
        const float u = (x - refu) * c;
        const float e = ex2_fast(u);
        z2 = f2_add(z2, f2_make(e, 0.f));
        if constexpr (ENT) w2 = f2_fma(f2_make(e, 0.f), f2_make(fmaxf(u, -1e30f), 0.f), w2);
    }
};

// The sums of several threads (or blocks), joined about the larger reference.  Symmetric in its
// arguments, so a butterfly leaves the same bits in every lane.
struct RowTotal {
    float ref, z, w;
};
__device__ __forceinline__ RowTotal total_about(RowTotal a, float m, float c) {
    if (a.ref == m) return a;
    if (a.ref == -INFINITY) return {m, a.z, 0.f};  // z is 0, or NaN
    const float d = (a.ref - m) * c;
    const float f = ex2_fast(d);
    return {m, __fmul_rn(f, a.z), __fmul_rn(f, __fmaf_rn(a.z, fmaxf(d, -1e30f), a.w))};
}
__device__ __forceinline__ RowTotal total_join(RowTotal a, RowTotal b, float c) {
    const float m = fmaxf(a.ref, b.ref);
    a = total_about(a, m, c);
    b = total_about(b, m, c);
    return {m, __fadd_rn(a.z, b.z), __fadd_rn(a.w, b.w)};
}
__device__ __forceinline__ RowTotal total_xor(RowTotal a, int o) {
    return {__shfl_xor_sync(kFullMask, a.ref, o), __shfl_xor_sync(kFullMask, a.z, o),
            __shfl_xor_sync(kFullMask, a.w, o)};
}

// A block's threads' sums joined, the same bits in every thread.  `sh`: one RowTotal a warp;
// the caller synchronises before the next use of it.
__device__ __forceinline__ RowTotal block_total(RowTotal a, float c, RowTotal* sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = total_join(a, total_xor(a, o), c);
    const int nw = (int)blockDim.x >> 5;
    if (nw == 1) return a;
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = a;
    __syncthreads();
    const int lane = (int)threadIdx.x & 31;
    a = lane < nw ? sh[lane] : RowTotal{-INFINITY, 0.f, 0.f};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = total_join(a, total_xor(a, o), c);
    return a;
}

}  // namespace lnk
