// ckpt8.cuh -- the 8-bit checkpoint's format on the device.
//
// 32 columns of a row (a block; the last one of a row may be shorter) are kept as integers q in
// -127 .. 127 and one byte k that stands for the step 2^(k - 127): x is taken back as q 2^(k - 127).
// The step is the least power of two for which the block's largest magnitude rounds to at most 127,
// 2^-126 at least.  With amax = f 2^E, 1 <= f < 2, that is 2^(E - 6) for f < 127.5 / 64 and 2^(E - 5)
// from there (127.5 itself would round to the even 128), so that k falls out of amax's bits: adding
// 2^16 to them carries into the exponent exactly from f = 127.5 / 64 = 1 + 127 / 128 on.  A power of two
// makes quotient and product exact, so that rounding q (to nearest, ties to even) is the one error: at
// most half a step, amax / 127 at most for normal numbers; and what a checkpoint stands for fits bf16
// exactly.  2^121 is the largest step (64 2^122 is no fp32 number): magnitudes of 127.5 2^121 and more are held to
// 127 2^121.  A block that holds an infinity or a NaN has k = 255 and q = 0: 0 times the infinity that
// 255 << 23 is gives NaN, so that such a block comes back as NaN throughout.
#pragma once

#include "ln_device.cuh"

namespace lnk {
namespace {

constexpr int kCkptBlock = 32;
constexpr uint32_t kCkptLargest = 248;  // k of the largest step

__host__ __device__ constexpr int ckpt_blocks(int cols) { return (cols + kCkptBlock - 1) / kCkptBlock; }

// k from the bits of the largest magnitude (an integer maximum of magnitudes' bits: NaN above infinity).
__device__ __forceinline__ uint32_t ckpt_byte(uint32_t amax) {
    return amax >= 0x7f800000u ? 255u : max((amax + 0x10000u) >> 23, 7u) - 6u;
}
// 1 / step for k of 1 .. 248 (for 255 the integers are not used).
__device__ __forceinline__ float ckpt_inverse(uint32_t k) { return __uint_as_float((254u - k) << 23); }
__device__ __forceinline__ float ckpt_step(uint32_t k) { return __uint_as_float(k << 23); }

// Adding 1.5 * 2^23 rounds to an integer (nearest, ties to even) and leaves it in the low bits.
constexpr float kRounder = 12582912.0f;

__device__ __forceinline__ uint32_t ckpt_pack4(f2 a, f2 b, f2 inv) {
    const f2 r = f2_splat(kRounder);
    const f2 p = f2_fma(a, inv, r), q = f2_fma(b, inv, r);  // the product is exact
    const uint32_t lo = __byte_perm(__float_as_uint(f2_lo(p)), __float_as_uint(f2_hi(p)), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(f2_lo(q)), __float_as_uint(f2_hi(q)), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}

// Four integers as floats: q + 128 in the low byte of 2^23 is 2^23 + 128 + q.
__device__ __forceinline__ void ckpt_integers4(uint32_t w, f2& a, f2& b) {
    w ^= 0x80808080u;
    const f2 off = f2_splat(-8388736.0f);
    a = f2_add(f2_make(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440)),
                       __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7441))), off);
    b = f2_add(f2_make(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7442)),
                       __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7443))), off);
}

// As the values they stand for.
__device__ __forceinline__ void ckpt_unpack4(uint32_t w, f2 step, f2& a, f2& b) {
    ckpt_integers4(w, a, b);
    a = f2_mul(a, step);
    b = f2_mul(b, step);
}

// The largest magnitude's bits over groups of LANES lanes' vectors of T (bf16: two columns of maxima at a time).
template <typename T, int LANES>
__device__ __forceinline__ uint32_t magnitude(const uint4& u) {
    if constexpr (sizeof(T) == 2) {
        uint32_t m = __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu),
                              __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(kFullMask, m, o));
        return max(m << 16, m & 0xffff0000u);
    } else {
        uint32_t m = max(max(u.x & 0x7fffffffu, u.y & 0x7fffffffu), max(u.z & 0x7fffffffu, u.w & 0x7fffffffu));
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) m = max(m, __shfl_xor_sync(kFullMask, m, o));
        return m;
    }
}

// A warp keeps 32 vectors of 16 bytes of a row: lane l has columns col .. col + V - 1 (col = first + l V,
// first a multiple of 32), as they are stored in T, zeros past the row's last column.  q and k: the row's
// integers (whole blocks) and bytes; columns of past and more are not kept.  Called by all lanes.
template <typename T>
__device__ __forceinline__ void ckpt_keep(const uint4& u, int col, int past, int8_t* q, uint8_t* k) {
    constexpr int V = Io<T>::kVec;
    uint32_t byte = ckpt_byte(magnitude<T, kCkptBlock / V>(u));
    if (col >= past) return;
    f2 v[Pairs<T>::kPairs];
    Pairs<T>::unpack(u, v);
    if (byte == kCkptLargest + 1) {
        byte = kCkptLargest;
        const float most = 127.f * ckpt_step(kCkptLargest);
#pragma unroll
        for (int h = 0; h < Pairs<T>::kPairs; ++h)
            v[h] = f2_make(fminf(fmaxf(f2_lo(v[h]), -most), most), fminf(fmaxf(f2_hi(v[h]), -most), most));
    }
    const f2 inv = f2_splat(ckpt_inverse(byte));
    if constexpr (V == 8) {
        uint2 w = make_uint2(ckpt_pack4(v[0], v[1], inv), ckpt_pack4(v[2], v[3], inv));
        if (byte == 255u) w = make_uint2(0u, 0u);
        *reinterpret_cast<uint2*>(q + col) = w;
    } else {
        *reinterpret_cast<uint32_t*>(q + col) = byte == 255u ? 0u : ckpt_pack4(v[0], v[1], inv);
    }
    if (col % kCkptBlock == 0) k[col / kCkptBlock] = (uint8_t)byte;
}

// The integers of V columns from a multiple of V.
template <typename T>
struct CkptRaw {
    static constexpr int kWords = Io<T>::kVec / 4;
    uint32_t w[kWords];
    uint32_t k;

    __device__ __forceinline__ void load(const int8_t* q, const uint8_t* kk, int col) {
        if constexpr (kWords == 2) {
            const uint2 u = __ldcs(reinterpret_cast<const uint2*>(q + col));
            w[0] = u.x;
            w[1] = u.y;
        } else {
            w[0] = __ldcs(reinterpret_cast<const uint32_t*>(q + col));
        }
        k = __ldg(kk + col / kCkptBlock);
    }
    __device__ __forceinline__ void values(f2 (&v)[Pairs<T>::kPairs]) const {
        const f2 step = f2_splat(ckpt_step(k));
#pragma unroll
        for (int i = 0; i < kWords; ++i) ckpt_unpack4(w[i], step, v[2 * i], v[2 * i + 1]);
    }
    // The integers, from where they start (shared memory, or global).
    __device__ __forceinline__ void take(const void* q) {
        if constexpr (kWords == 2) {
            const uint2 u = *reinterpret_cast<const uint2*>(q);
            w[0] = u.x;
            w[1] = u.y;
        } else {
            w[0] = *reinterpret_cast<const uint32_t*>(q);
        }
    }
    // The values plus c, each rounded once (the product is exact).
    __device__ __forceinline__ void values(f2 (&v)[Pairs<T>::kPairs], f2 c) const {
        const f2 step = f2_splat(ckpt_step(k));
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            ckpt_integers4(w[i], v[2 * i], v[2 * i + 1]);
            v[2 * i] = f2_fma(v[2 * i], step, c);
            v[2 * i + 1] = f2_fma(v[2 * i + 1], step, c);
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
        k = 0;
    }
    // Zeros from the count-th column on.
    __device__ __forceinline__ void first(int count) {
        if (count <= 0) k = 0;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const int left = count - 4 * i;
            w[i] &= left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
        }
    }
};

}  // namespace
}  // namespace lnk
