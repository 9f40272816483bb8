// vocab.cuh -- device-side building blocks of the operators over rows of logits
// (logprobs.cu, distill.cu): a row as 16-byte vectors and loose ends, and the running
// softmax sums of a row.
#pragma once

#include <math.h>

#include "ln_device.cuh"

namespace lnk {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// A row of V logits at any element-aligned address: `head` loose elements up to the first boundary of
// BYTES (16, or 32 where vectors are taken in pairs), `nvec` 16-byte vectors, `tail` loose elements
// behind them.  Rows of an odd length one after another start at a different place of a vector each;
// cutting every row at its own boundaries keeps all but a few elements on wide accesses.
template <typename T, int BYTES = 16>
struct RowCut {
    int head, nvec, tail;
    __device__ __forceinline__ RowCut(const T* row, int V) {
        constexpr int kVec = Io<T>::kVec, kUnit = BYTES / (int)sizeof(T);
        const int mis = (int)(reinterpret_cast<uintptr_t>(row) & (BYTES - 1u)) / (int)sizeof(T);
        head = min(V, (kUnit - mis) % kUnit);
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

// A batch: kBatch vectors of one thread, loaded together.
constexpr int kBatch = 4;

// Vectors that hold nothing: every value -inf.
template <typename T>
__device__ __forceinline__ uint4 no_logits() {
    const unsigned w = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
    return make_uint4(w, w, w, w);
}

// Vectors v0, v0 + step, ... below `end` of a row's slice; what lies behind it holds nothing.
template <typename T>
__device__ __forceinline__ void load_batch(uint4 (&u)[kBatch], const uint4* xv, int v0, int step, int end) {
    if (v0 + (kBatch - 1) * step < end) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) u[k] = __ldcg(xv + v0 + k * step);
    } else {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int v = v0 + k * step;
            u[k] = v < end ? __ldcg(xv + v) : no_logits<T>();
        }
    }
}

// The same with a batch of two pairs of neighbouring vectors, the second pair 2 * step behind the first,
// each pair one 256-bit access (v0 even, the row cut at 32 bytes): a thread's vectors fill whole
// 32-byte sectors, which counts when few of them are read again.
__device__ __forceinline__ int pair_vector(int v0, int step, int k) { return v0 + (k >> 1) * 2 * step + (k & 1); }
template <typename T>
__device__ __forceinline__ void load_pairs(uint4 (&u)[kBatch], const uint4* xv, int v0, int step, int end) {
    static_assert(kBatch == 4, "two pairs");
    if (v0 + 2 * step + 1 < end) {
#pragma unroll
        for (int k = 0; k < kBatch; k += 2) {
            uint4 &a = u[k], &b = u[k + 1];
            asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                         : "l"(xv + v0 + k * step));
        }
    } else {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int v = pair_vector(v0, step, k);
            u[k] = v < end ? __ldcg(xv + v) : no_logits<T>();
        }
    }
}

// The largest value of N vectors in fp32 (exact).  NAN_TOO: NaN if there is one, else NaN loses
// against a number.
template <typename T, bool NAN_TOO, int N>
__device__ __forceinline__ float largest(const uint4 (&u)[N]) {
    if constexpr (sizeof(T) == 2) {
        auto two = [](unsigned a, unsigned b) {
            unsigned m;
            if constexpr (NAN_TOO)
                asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
            else
                asm("max.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
            return m;
        };
        unsigned m = two(two(u[0].x, u[0].y), two(u[0].z, u[0].w));
#pragma unroll
        for (int k = 1; k < N; ++k) m = two(m, two(two(u[k].x, u[k].y), two(u[k].z, u[k].w)));
        m = two(m, (m >> 16) | (m << 16));
        return __uint_as_float(m << 16);
    } else {
        auto three = [](float a, float b, float c) {
            float m;
            if constexpr (NAN_TOO)
                asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
            else
                asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
            return m;
        };
        auto f = [](unsigned a) { return __uint_as_float(a); };
        float m = three(f(u[0].w), f(u[0].x), three(f(u[0].y), f(u[0].z), f(u[0].w)));
#pragma unroll
        for (int k = 1; k < N; ++k)
            m = three(m, f(u[k].x), three(f(u[k].y), f(u[k].z), f(u[k].w)));
        return m;
    }
}
template <typename T>
__device__ __forceinline__ float vector_max(const uint4& u) {
    const uint4 one[1] = {u};
    return largest<T, false>(one);
}

// The differences of a vector's values to r, as fp32 pairs (exact for bf16 values near r; one
// rounding otherwise).
template <typename T>
__device__ __forceinline__ void less(const uint4& u, float r, f2 (&d)[Pairs<T>::kPairs]) {
    if constexpr (sizeof(T) == 2) {
        // bf16 - fp32 in one instruction a value, without unpacking it first (sm_100 family).
        const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            float lo, hi;
            asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
                "sub.rn.f32.bf16 %0, l, %3;\n\tsub.rn.f32.bf16 %1, h, %3;\n\t}"
                : "=f"(lo), "=f"(hi)
                : "r"(w[h]), "f"(r));
            d[h] = f2_make(lo, hi);
        }
    } else {
        const f2 r2 = f2_splat(r);
        Pairs<T>::unpack(u, d);
#pragma unroll
        for (int h = 0; h < Pairs<T>::kPairs; ++h) d[h] = f2_sub(d[h], r2);
    }
}

// How many values of a batch are above x.
template <typename T>
__device__ __forceinline__ int count_above(const uint4 (&u)[kBatch], float x) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        float f[Io<T>::kVec];
        Io<T>::unpack(u[k], f);
#pragma unroll
        for (int j = 0; j < Io<T>::kVec; ++j) n += f[j] > x;
    }
    return n;
}

// Running sums of a softmax over the values seen so far, about a reference value `ref`:
//   u = (x - ref) * c,  z = sum 2^u,  w = sum 2^u u          (c = scale * log2 e).
// The reference is a value of the row, at most kSlack / c below the largest one: it is replaced,
// and the sums rescaled, only when a value exceeds it by more than that.  A plain running maximum
// moves for some lane of a warp in almost every step of a row of a few thousand values; this one
// moves once or twice a row, and log z - ln 2 w / z has terms of at most kSlack more to cancel.
// ref = -inf: no value above -inf yet; u is then taken about 0, so that -inf adds nothing and a
// NaN still reaches z.  The differences x - ref are taken before the product with c: a value next
// to the reference keeps its exact distance whatever the size of both.
constexpr float kSlack = 8.f;

template <bool ENT>
struct RowSums {
    float ref, refu;  // refu: ref, or 0 while ref is -inf
    float lim;        // values up to it need no new reference (see() decides about the others)
    f2 z2, w2;
    __device__ __forceinline__ void clear() {
        ref = lim = -INFINITY;
        refu = 0.f;
        z2 = f2_splat(0.f);
        w2 = f2_splat(0.f);
    }
    // See a value m (not NaN): move the reference there if it lies too far above.
    __device__ __forceinline__ void see(float m, float c) {
        if (!(m > ref) || (m - ref) * c <= kSlack) return;
        if (ref != -INFINITY) {
            const float d = (ref - m) * c;
            const f2 f = f2_splat(ex2_fast(d));
            if constexpr (ENT) w2 = f2_mul(f, f2_fma(z2, f2_splat(fmaxf(d, -1e30f)), w2));
            z2 = f2_mul(f, z2);
        }
        ref = refu = m;
        lim = fminf(m + kSlack / c, 3.402823466e38f);
    }
    // One vector's terms.  0 * -inf is no term of w: the exponent is held at a value whose weight is 0 too.
    template <typename T>
    __device__ __forceinline__ void add(const uint4& v, f2 c2) {
        constexpr int H = Pairs<T>::kPairs;
        f2 d[H];
        less<T>(v, refu, d);
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const f2 u = f2_mul(d[h], c2);
            const f2 e = f2_make(ex2_fast(f2_lo(u)), ex2_fast(f2_hi(u)));
            z2 = f2_add(z2, e);
            if constexpr (ENT)
                w2 = f2_fma(e, f2_make(fmaxf(f2_lo(u), -1e30f), fmaxf(f2_hi(u), -1e30f)), w2);
        }
    }
    // A batch's largest value, NaN left out, after seeing it; -inf: there is nothing to add.
    template <typename T>
    __device__ __forceinline__ float see_batch(const uint4 (&u)[kBatch], float c) {
        float m = largest<T, true>(u);
        if (!(m <= lim)) {  // rare: perhaps a new reference, or NaN
            if (m != m) {
                m = largest<T, false>(u);
                z2 = f2_splat(__int_as_float(0x7fc00000));  // no distribution
            }
            see(m, c);
        }
        return m;
    }
    // Add the batch that see_batch() has seen.
    template <typename T>
    __device__ __forceinline__ void add_batch(const uint4 (&u)[kBatch], f2 c2) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) add<T>(u[k], c2);
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
__device__ __forceinline__ float warp_max(float v) {
    float m;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}
// A warp's sums joined, the same bits in every lane: all are taken about the largest reference, and
// then only added.
__device__ __forceinline__ RowTotal warp_total(RowTotal a, float c) {
    a = total_about(a, warp_max(a.ref), c);
    warp_sum2(a.z, a.w);
    return a;
}
// A block's threads' sums joined, the same bits in every thread.  `sh`: one RowTotal a warp;
// the caller synchronises before the next use of it.
__device__ __forceinline__ RowTotal block_total(RowTotal a, float c, RowTotal* sh) {
    a = warp_total(a, c);
    const int nw = (int)blockDim.x >> 5;
    if (nw == 1) return a;
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = a;
    __syncthreads();
    const int lane = (int)threadIdx.x & 31;
    a = lane < nw ? sh[lane] : RowTotal{-INFINITY, 0.f, 0.f};
    return warp_total(a, c);
}

// ---------------------------------------------------------------------------------------
// Thread-block clusters: the blocks of a cluster run at the same time, and write to one another's
// shared memory once all of them have arrived at the cluster's barrier for the first time.
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_blocks() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// The address, in block `rank`'s shared memory, of what is at p in this block's.
__device__ __forceinline__ uint32_t in_block(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void st_cluster_f32(uint32_t a, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
// Asynchronous stores to another block, whose mbarrier at `bar` counts their bytes.
__device__ __forceinline__ void send2(uint32_t a, float x, float y, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(a),
                 "r"(__float_as_uint(x)), "r"(__float_as_uint(y)), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void send4(uint32_t a, float x, float y, float z, uint32_t bar) {
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(a),
        "r"(__float_as_uint(x)), "r"(__float_as_uint(y)), "r"(__float_as_uint(z)), "r"(0u), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void st_cluster_u64(uint32_t a, unsigned long long v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

}  // namespace lnk
