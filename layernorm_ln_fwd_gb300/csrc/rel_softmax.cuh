// rel_softmax.cuh -- softmax of attention scores with a learned relative position bias, and its gradients.
//
// For sequence b, head h, query i at position p = q_pos[b] + i and key j at distance d = j - p:
//   z_j = scale x_j + table[bucket(d), h] + mask_j,   y = softmax(z) over the keys that take part,
//   dS = y (dy - sum dy y),  dx = scale dS,  dtable[k, h] = sum of dS over b, i and the j of bucket k.
// A key of lens[b] or more, or behind its query where the call is causal, takes no part, and nor does one
// whose z is -inf: y = 0 there, and a row with nothing left is 0 throughout.
//
// Buckets.  Beyond the last edge every distance of a side has one bucket, so that a block needs the table
// at a window of distances only, spread out in shared memory once for the block's queries (all of one
// sequence and head): 2 * 91 + 1 entries for 32 buckets up to 128, whatever the row's length.  Columns
// outside the window take its end value from a register.  The gradient goes the same way back: each
// warp adds dS into a window of its own by distance, with loads and stores (a row meets each distance once,
// rows follow one another), sums both far ends in registers, and the block adds the windows up and cuts them
// into buckets at its end.  Nothing is atomic; the order of all sums is fixed by the sizes.
//
// Entry t of a window is at t + t / V: lanes read V consecutive entries each, V apart, and the spare word
// behind every V moves them to different banks.
//
// A row is held in registers by 1 to 16 warps (a team), read once and written once; what a causal row or a
// short sequence leaves out is not read.  Rows of more columns than 16 warps hold are gone through twice.
// Bound by memory: see the figures at the kernels.
#pragma once

#include <limits.h>

#include <algorithm>
#include <type_traits>

#include "ckpt8.cuh"
#include "rel_ops.h"
#include "row_io.cuh"

namespace lnk {
namespace {

constexpr float kRelLog2e = 1.4426950408889634f;
constexpr int kRelFar = 1 << 30;  // positions are held to this: every bucket ends long before

struct RelParams {
    const void* a;
    const void* y;
    void* out;
    int64_t lda, ldy, ldo, ldm;
    int8_t* q;
    uint8_t* k;
    const void* mask;
    int64_t mask_rows;
    const void* table;
    int table_f32;
    const int* lens;
    const int* q_pos;
    int H, Lq, Lk, rows, chunks, causal;
    float scale;
    Extent ea, ey, em;
    float* part;
    RelBuckets bk;
};

// What a block works on.
struct RelBlock {
    int64_t row0;    // its first row in the call
    int b, h;
    int i0, i1;      // queries
    int len;         // the sequence's keys
    int at;          // position of the sequence's query 0
    int dlo, dhi;    // the window's distances
    int wlen;        // its entries: V more at either end
};

__device__ __forceinline__ int rel_bucket(const RelBuckets& bk, const int* edge, int d) {
    const int n = d <= 0 ? -d : bk.both ? d : 0;
    int lo = 0, hi = bk.n;  // the number of edges at or below n
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (edge[mid] <= n)
            lo = mid + 1;
        else
            hi = mid;
    }
    return d > 0 && bk.both ? lo + bk.n + 1 : lo;
}

template <int V>
__device__ __forceinline__ RelBlock rel_block(const RelParams& p) {
    RelBlock r;
    const int m = (int)blockIdx.x / p.chunks, c = (int)blockIdx.x - m * p.chunks;
    r.b = m / p.H;
    r.h = m - r.b * p.H;
    r.i0 = c * p.rows;
    r.i1 = min(p.Lq, r.i0 + p.rows);
    r.row0 = (int64_t)m * p.Lq + r.i0;
    r.len = p.lens ? min(max(__ldg(p.lens + r.b), 0), p.Lk) : p.Lk;
    r.at = p.q_pos ? min(max(__ldg(p.q_pos + r.b), -kRelFar), kRelFar) : 0;
    const int last = p.bk.n ? p.bk.edge[p.bk.n - 1] : 1;  // at least 1: d > 0 and d <= 0 have two ends
    const int hi = p.bk.both ? last : 0;
    r.dlo = min(max(-(r.at + r.i1 - 1), -last), hi);
    r.dhi = min(max(p.Lk - 1 - (r.at + r.i0), r.dlo), hi);
    r.wlen = r.dhi - r.dlo + 1 + 2 * V;
    return r;
}

template <int V>
__device__ __forceinline__ int spread(int t) {
    return t + (int)((unsigned)t / V);  // t >= 0
}

// Keys of query i that take part: the first n columns.
__device__ __forceinline__ int rel_keys(const RelParams& p, const RelBlock& r, int i) {
    return p.causal ? min(r.len, max(r.at + i + 1, 0)) : r.len;
}

template <int W, int TEAMS>
__device__ __forceinline__ void team_sync(int team) {
    if constexpr (TEAMS == 1) {
        __syncthreads();
    } else {
        asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(W * 32) : "memory");
    }
}

__device__ __forceinline__ float rel_warp_max(float a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(kFullMask, a, o));
    return a;
}
__device__ __forceinline__ float rel_warp_sum(float a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(kFullMask, a, o);
    return a;
}

// exp2((m - M) log2 e), the factor from sums taken against m to those against M >= m; 1 for a sum that
// met nothing (m = -inf), which is 0, or NaN.
__device__ __forceinline__ float rel_factor(float m, float M) {
    return m == -INFINITY ? 1.f : ex2_fast((m - M) * kRelLog2e);
}

// ---------------------------------------------------------------------------------------
// Forward.
// ---------------------------------------------------------------------------------------

// The scores z of vector `col` of a row with n keys that take part: -inf elsewhere.  win: the bias's window
// (lo, hi: its end values), t0: the entry of column 0.
template <typename T>
__device__ __forceinline__ void rel_scores(const uint4& raw, const T* mrow, const Extent& em, int col, int n,
                                           int t0, int wlen, const float* win, float lo, float hi, f2 scale,
                                           f2 (&z)[Pairs<T>::kPairs]) {
    constexpr int V = Io<T>::kVec, H = Pairs<T>::kPairs;
    f2 x[H];
    Pairs<T>::unpack(raw, x);
    const int t = t0 + col;  // entries t .. t + V - 1; those below 1 and from wlen - V on are the ends
    if (t <= 1) {
        const f2 b = f2_splat(lo);
#pragma unroll
        for (int h = 0; h < H; ++h) z[h] = f2_fma(scale, x[h], b);
    } else if (t >= wlen - V) {
        const f2 b = f2_splat(hi);
#pragma unroll
        for (int h = 0; h < H; ++h) z[h] = f2_fma(scale, x[h], b);
    } else {
        const int c = t & (V - 1);
        const float* w = win + spread<V>(t);
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const float b0 = w[2 * h + (c + 2 * h >= V)], b1 = w[2 * h + 1 + (c + 2 * h + 1 >= V)];
            z[h] = f2_fma(scale, x[h], f2_make(b0, b1));
        }
    }
    if (mrow) {
        f2 mv[H];
        Pairs<T>::unpack(load_columns<T>(mrow, col, n, em), mv);
#pragma unroll
        for (int h = 0; h < H; ++h) {  // a mask of -inf removes a key whatever its score is
            const f2 s = f2_add(z[h], mv[h]);
            z[h] = f2_make(f2_lo(mv[h]) == -INFINITY ? -INFINITY : f2_lo(s),
                           f2_hi(mv[h]) == -INFINITY ? -INFINITY : f2_hi(s));
        }
    }
    if (col + V > n) {
#pragma unroll
        for (int h = 0; h < H; ++h)
            z[h] = f2_make(col + 2 * h < n ? f2_lo(z[h]) : -INFINITY,
                           col + 2 * h + 1 < n ? f2_hi(z[h]) : -INFINITY);
    }
}

// y of a vector: e c, zeros from column n on, stored (and kept in 8 bits).  Called by all lanes.
template <typename T, bool CKPT>
__device__ __forceinline__ void rel_put(const RelParams& p, T* yrow, int8_t* qrow, uint8_t* krow, int col, int n,
                                        const f2 (&e)[Pairs<T>::kPairs], float c) {
    constexpr int V = Io<T>::kVec, H = Pairs<T>::kPairs;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (col < n) {
        f2 o[H];
        const f2 c2 = f2_splat(c);
#pragma unroll
        for (int h = 0; h < H; ++h) o[h] = f2_mul(e[h], c2);
        u = Pairs<T>::pack(o);
        if (col + V > n) u = first_of<T>(u, n - col);
    }
    store_columns<T>(yrow, col, p.Lk, u);
    if constexpr (CKPT) ckpt_keep<T>(u, col, ckpt_blocks(p.Lk) * kCkptBlock, qrow, krow);
}

// W warps hold a row, NV vectors a lane (vector (k W + w) 32 + l); TEAMS rows at a time.  LOOP: rows of any
// length, in tiles of that size, twice.
template <typename T, int W, int TEAMS, int NV, bool LOOP, bool CKPT>
__global__ void __launch_bounds__(W * TEAMS * 32) rel_fwd_kernel(const __grid_constant__ RelParams p) {
    constexpr int V = Io<T>::kVec, H = Pairs<T>::kPairs;
    constexpr int kThreads = W * TEAMS * 32;
    constexpr int kTile = W * NV * 32 * V;
    extern __shared__ float win[];
    __shared__ int edge[kRelMaxEdges];
    __shared__ float red[2][TEAMS][2][W];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int team = warp / W, wt = warp - team * W;
    for (int i = tid; i < p.bk.n; i += kThreads) edge[i] = p.bk.edge[i];
    pdl_enter();
    const RelBlock r = rel_block<V>(p);
    __syncthreads();
    for (int t = tid; t < r.wlen; t += kThreads) {
        const int d = min(max(r.dlo + t - V, r.dlo), r.dhi);
        const int at = rel_bucket(p.bk, edge, d) * p.H + r.h;
        win[spread<V>(t)] = p.table_f32 ? __ldg(static_cast<const float*>(p.table) + at)
                                        : __bfloat162float(static_cast<const __nv_bfloat16*>(p.table)[at]);
    }
    __syncthreads();
    const float lo = win[0], hi = win[spread<V>(r.wlen - 1)];
    const f2 scale = f2_splat(p.scale), l2 = f2_splat(kRelLog2e);
    const int padded = CKPT ? ckpt_blocks(p.Lk) * kCkptBlock : p.Lk;
    int parity = 0;
    for (int i = r.i0 + team; i < r.i1; i += TEAMS, parity ^= 1) {
        const int64_t row = r.row0 + (i - r.i0);
        const int n = rel_keys(p, r, i);
        const T* x = static_cast<const T*>(p.a) + row * p.lda;
        T* y = static_cast<T*>(p.out) + row * p.ldo;
        const T* mrow = p.mask ? static_cast<const T*>(p.mask) + (row % p.mask_rows) * p.ldm : nullptr;
        int8_t* qrow = CKPT ? p.q + row * padded : nullptr;
        uint8_t* krow = CKPT ? p.k + row * (padded / kCkptBlock) : nullptr;
        const int t0 = V - r.dlo - (r.at + i);  // window entry of column 0
        f2 z[NV][H];
        float m = -INFINITY, s = 0.f;
        const int tiles = LOOP ? (n + kTile - 1) / kTile : 1;
        auto scores = [&](int base) {
            uint4 raw[NV];
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = base + ((k * W + wt) * 32 + lane) * V;
                if (col < n) raw[k] = load_columns<T>(x, col, n, p.ea);
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = base + ((k * W + wt) * 32 + lane) * V;
                if (col < n) {
                    rel_scores<T>(raw[k], mrow, p.em, col, n, t0, r.wlen, win, lo, hi, scale, z[k]);
                } else {
#pragma unroll
                    for (int h = 0; h < H; ++h) z[k][h] = f2_splat(-INFINITY);
                }
            }
        };
        // z becomes exp(z - ref).
        auto weights = [&](float ref) {
            const f2 nr = f2_splat(-ref);
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const f2 t = f2_mul(f2_add(z[k][h], nr), l2);
                    z[k][h] = f2_make(ex2_fast(f2_lo(t)), ex2_fast(f2_hi(t)));
                }
        };
        for (int tile = 0; tile < tiles; ++tile) {
            scores(tile * kTile);
            float mt = -INFINITY;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int h = 0; h < H; ++h) mt = fmaxf(mt, fmaxf(f2_lo(z[k][h]), f2_hi(z[k][h])));
            mt = rel_warp_max(mt);
            if constexpr (LOOP) {
                mt = fmaxf(mt, m);
                s = s * rel_factor(m, mt);
            }
            m = mt;
            weights(m == -INFINITY ? 0.f : m);
            f2 acc = f2_splat(0.f);
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int h = 0; h < H; ++h) acc = f2_add(acc, z[k][h]);
            s += f2_lo(acc) + f2_hi(acc);
        }
        s = rel_warp_sum(s);
        float c;
        if constexpr (W == 1) {
            c = s == 0.f ? 0.f : 1.f / s;
        } else {  // the warps' (max, sum) meet once
            if (lane == 0) {
                red[parity][team][0][wt] = m;
                red[parity][team][1][wt] = s;
            }
            team_sync<W, TEAMS>(team);
            float M = -INFINITY, S = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) M = fmaxf(M, red[parity][team][0][w]);
#pragma unroll
            for (int w = 0; w < W; ++w) S += red[parity][team][1][w] * rel_factor(red[parity][team][0][w], M);
            c = S == 0.f ? 0.f : rel_factor(m, M) / S;
        }
        const int out_tiles = LOOP ? (padded + kTile - 1) / kTile : 1;
        for (int tile = 0; tile < out_tiles; ++tile) {
            const int base = tile * kTile;
            if constexpr (LOOP) {
                scores(base);
                weights(m == -INFINITY ? 0.f : m);
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int first = base + (k * W + wt) * 32 * V;
                if (first < p.Lk) rel_put<T, CKPT>(p, y, qrow, krow, first + lane * V, n, z[k], c);
            }
        }
    }
}

// ---------------------------------------------------------------------------------------
// Backward.
// ---------------------------------------------------------------------------------------

// A row's probabilities: stored in T, or in 8 bits.
template <typename T, bool CKPT>
struct Probs {
    uint4 u;
    __device__ __forceinline__ void load(const RelParams& p, const T* yrow, const int8_t*, const uint8_t*, int col,
                                         int n) {
        u = load_columns<T>(yrow, col, n, p.ey);
    }
    __device__ __forceinline__ void first(int count) { u = first_of<T>(u, count); }
    __device__ __forceinline__ void values(f2 (&v)[Pairs<T>::kPairs]) const { Pairs<T>::unpack(u, v); }
};
template <typename T>
struct Probs<T, true> {
    CkptRaw<T> r;
    __device__ __forceinline__ void load(const RelParams&, const T*, const int8_t* qrow, const uint8_t* krow, int col,
                                         int) {
        r.load(qrow, krow, col);
    }
    __device__ __forceinline__ void first(int count) { r.first(count); }
    __device__ __forceinline__ void values(f2 (&v)[Pairs<T>::kPairs]) const { r.values(v); }
};

// 0 where y is, whatever g is.
__device__ __forceinline__ f2 where_weight(f2 y, f2 g) {
    return f2_make(f2_lo(y) == 0.f ? 0.f : f2_lo(g), f2_hi(y) == 0.f ? 0.f : f2_hi(g));
}

template <typename T, int W, int TEAMS, int NV, bool LOOP, bool CKPT>
__global__ void __launch_bounds__(W * TEAMS * 32) rel_bwd_kernel(const __grid_constant__ RelParams p) {
    constexpr int V = Io<T>::kVec, H = Pairs<T>::kPairs;
    constexpr int kThreads = W * TEAMS * 32;
    constexpr int kTile = W * NV * 32 * V;
    extern __shared__ float win[];
    __shared__ int edge[kRelMaxEdges];
    __shared__ float red[2][TEAMS][W];
    __shared__ float far_sums[W * TEAMS][2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int team = warp / W, wt = warp - team * W;
    for (int i = tid; i < p.bk.n; i += kThreads) edge[i] = p.bk.edge[i];
    pdl_enter();
    const RelBlock r = rel_block<V>(p);
    const int stride = spread<V>(r.wlen - 1) + 1;
    float* mine = win + team * stride;
    const bool sums = p.part != nullptr;
    if (sums)
        for (int t = tid; t < TEAMS * stride; t += kThreads) win[t] = 0.f;
    __syncthreads();
    const f2 scale = f2_splat(p.scale);
    f2 below = f2_splat(0.f), above = f2_splat(0.f);  // dS of the far ends
    const int padded = ckpt_blocks(p.Lk) * kCkptBlock;
    int parity = 0;
    for (int i = r.i0 + team; i < r.i1; i += TEAMS) {
        const int64_t row = r.row0 + (i - r.i0);
        const int n = rel_keys(p, r, i);
        const T* dy = static_cast<const T*>(p.a) + row * p.lda;
        const T* yrow = CKPT ? nullptr : static_cast<const T*>(p.y) + row * p.ldy;
        const int8_t* qrow = CKPT ? p.q + row * padded : nullptr;
        const uint8_t* krow = CKPT ? p.k + row * (padded / kCkptBlock) : nullptr;
        T* dx = static_cast<T*>(p.out) + row * p.ldo;
        const int t0 = V - r.dlo - (r.at + i);
        uint4 g[NV];
        Probs<T, CKPT> pr[NV];
        const int tiles = LOOP ? (n + kTile - 1) / kTile : 1;
        auto load = [&](int base) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = base + ((k * W + wt) * 32 + lane) * V;
                if (col < n) {
                    g[k] = load_columns<T>(dy, col, n, p.ea);
                    pr[k].load(p, yrow, qrow, krow, col, n);
                }
            }
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = base + ((k * W + wt) * 32 + lane) * V;
                if (col < n && col + V > n) {
                    g[k] = first_of<T>(g[k], n - col);
                    pr[k].first(n - col);
                }
            }
        };
        // sum dy y over the row; `careful`: without what a weight of 0 meets.
        auto row_sum = [&](auto careful) {
            float s = 0.f;
            for (int tile = 0; tile < tiles; ++tile) {
                if constexpr (LOOP) load(tile * kTile);
                f2 acc = f2_splat(0.f);
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int col = tile * kTile + ((k * W + wt) * 32 + lane) * V;
                    if (col >= n) continue;
                    f2 d[H], y[H];
                    Pairs<T>::unpack(g[k], d);
                    pr[k].values(y);
#pragma unroll
                    for (int h = 0; h < H; ++h)
                        acc = f2_fma(decltype(careful)::value ? where_weight(y[h], d[h]) : d[h], y[h], acc);
                }
                s += f2_lo(acc) + f2_hi(acc);
            }
            s = rel_warp_sum(s);
            if constexpr (W > 1) {
                if (lane == 0) red[parity][team][wt] = s;
                team_sync<W, TEAMS>(team);
                s = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w) s += red[parity][team][w];
                parity ^= 1;
            }
            return s;
        };
        if constexpr (!LOOP) load(0);
        float s = row_sum(std::false_type{});
        // A sum that is not finite (an infinite or NaN dy, perhaps at a key of weight 0, where it must
        // not count) is formed again without such keys.
        const bool careful = !(fabsf(s) < INFINITY);
        if (careful) s = row_sum(std::true_type{});
        const f2 s2 = f2_splat(s);
        const int out_tiles = LOOP ? (p.Lk + kTile - 1) / kTile : 1;
        for (int tile = 0; tile < out_tiles; ++tile) {
            const int base = tile * kTile;
            if constexpr (LOOP) load(base);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int first = base + (k * W + wt) * 32 * V, col = first + lane * V;
                if (first >= p.Lk) continue;
                uint4 u = make_uint4(0, 0, 0, 0);
                if (col < n) {
                    f2 d[H], y[H], o[H];
                    Pairs<T>::unpack(g[k], d);
                    pr[k].values(y);
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        d[h] = f2_mul(y[h], f2_sub(d[h], s2));
                        if (careful) d[h] = where_weight(y[h], d[h]);
                        o[h] = f2_mul(scale, d[h]);
                    }
                    u = Pairs<T>::pack(o);
                    if (col + V > n) u = first_of<T>(u, n - col);
                    if (sums) {
                        const int t = t0 + col;
                        if (t <= 1) {
#pragma unroll
                            for (int h = 0; h < H; ++h) below = f2_add(below, d[h]);
                        } else if (t >= r.wlen - V) {
#pragma unroll
                            for (int h = 0; h < H; ++h) above = f2_add(above, d[h]);
                        } else {
                            const int c = t & (V - 1);
                            float* w = mine + spread<V>(t);
                            float v[V];
#pragma unroll
                            for (int e = 0; e < V; ++e) v[e] = w[e + (c + e >= V)];
#pragma unroll
                            for (int h = 0; h < H; ++h) {
                                v[2 * h] += f2_lo(d[h]);
                                v[2 * h + 1] += f2_hi(d[h]);
                            }
#pragma unroll
                            for (int e = 0; e < V; ++e) w[e + (c + e >= V)] = v[e];
                        }
                    }
                }
                store_columns<T>(dx, col, p.Lk, u);
            }
        }
        if constexpr (W == 1) __syncwarp();  // the next row's entries are other lanes'
    }
    if (!sums) return;
    const float fb = rel_warp_sum(f2_lo(below) + f2_hi(below)), fa = rel_warp_sum(f2_lo(above) + f2_hi(above));
    if (lane == 0) {
        far_sums[warp][0] = fb;
        far_sums[warp][1] = fa;
    }
    __syncthreads();
    for (int t = tid; t < r.wlen; t += kThreads) {  // the teams' windows, and the far ends into the ends
        float v = 0.f;
        for (int k = 0; k < TEAMS; ++k) v += win[k * stride + spread<V>(t)];
        if (t == 0)
            for (int w = 0; w < W * TEAMS; ++w) v += far_sums[w][0];
        if (t == r.wlen - 1)
            for (int w = 0; w < W * TEAMS; ++w) v += far_sums[w][1];
        win[spread<V>(t)] = v;
    }
    __syncthreads();
    const int side = p.bk.n + 1, total = side * (p.bk.both ? 2 : 1);
    for (int k = warp; k < total; k += W * TEAMS) {
        // The bucket's distances a .. b, then the window's entries: with an end go the entries beyond it.
        const int j = k < side ? k : k - side;
        const int near = j ? edge[j - 1] : 0, far = j < p.bk.n ? edge[j] - 1 : INT_MAX;
        int a, b;
        if (k < side) {
            a = far == INT_MAX ? INT_MIN : -far;
            b = j == 0 && !p.bk.both ? INT_MAX : -near;
        } else {
            a = max(near, 1);
            b = far;
        }
        float v = 0.f;
        a = max(a, r.dlo);
        b = min(b, r.dhi);
        if (a <= b) {
            const int ta = a == r.dlo ? 0 : a - r.dlo + V, tb = b == r.dhi ? r.wlen - 1 : b - r.dlo + V;
            for (int t = ta + lane; t <= tb; t += 32) v += win[spread<V>(t)];
        }
        v = rel_warp_sum(v);
        if (lane == 0) p.part[(int64_t)blockIdx.x * total + k] = v;
    }
}

// ---------------------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------------------
struct RelShape {
    int W, teams, nv;
    bool loop;
};
// By capacity: 32 W nv vectors a row.
constexpr RelShape kRelShapes[] = {{1, 8, 1, false}, {1, 8, 2, false}, {1, 8, 4, false}, {2, 4, 4, false},
                                   {4, 2, 4, false}, {8, 1, 4, false}, {16, 1, 4, false}, {16, 1, 4, true},
                                   {1, 1, 2, false}, {8, 1, 1, false}, {8, 1, 2, false}};

template <typename T, bool BWD, bool CKPT, int W, int TEAMS, int NV, bool LOOP>
const void* rel_kernel_of() {
    if constexpr (BWD)
        return (const void*)rel_bwd_kernel<T, W, TEAMS, NV, LOOP, CKPT>;
    else
        return (const void*)rel_fwd_kernel<T, W, TEAMS, NV, LOOP, CKPT>;
}

template <typename T, bool BWD, bool CKPT>
const void* rel_kernel(int shape) {
    switch (shape) {
        case 0: return rel_kernel_of<T, BWD, CKPT, 1, 8, 1, false>();
        case 1: return rel_kernel_of<T, BWD, CKPT, 1, 8, 2, false>();
        case 2: return rel_kernel_of<T, BWD, CKPT, 1, 8, 4, false>();
        case 3: return rel_kernel_of<T, BWD, CKPT, 2, 4, 4, false>();
        case 4: return rel_kernel_of<T, BWD, CKPT, 4, 2, 4, false>();
        case 5: return rel_kernel_of<T, BWD, CKPT, 8, 1, 4, false>();
        case 6: return rel_kernel_of<T, BWD, CKPT, 16, 1, 4, false>();
        case 7: return rel_kernel_of<T, BWD, CKPT, 16, 1, 4, true>();
        case 8: return rel_kernel_of<T, BWD, CKPT, 1, 1, 2, false>();
        case 9: return rel_kernel_of<T, BWD, CKPT, 8, 1, 1, false>();
        case 10: return rel_kernel_of<T, BWD, CKPT, 8, 1, 2, false>();
        default: return nullptr;
    }
}

template <typename T, bool BWD>
cudaError_t launch_rel_t(const RelArgs& a, const RelPlan& plan, cudaStream_t stream, int* launches) {
    constexpr int V = Io<T>::kVec;
    *launches = 0;
    const RelShape& sh = kRelShapes[plan.shape];
    const bool ckpt = a.q != nullptr;
    const void* kern = ckpt ? rel_kernel<T, BWD, true>(plan.shape) : rel_kernel<T, BWD, false>(plan.shape);
    RelParams p;
    const int64_t rows = (int64_t)a.B * a.H * a.Lq;
    auto extent = [&](const void* t, int64_t n, int64_t ld) {
        const char* c = static_cast<const char*>(t);
        return Extent{c, c ? c + ((n - 1) * ld + a.Lk) * (int64_t)sizeof(T) : c};
    };
    p.a = a.a;
    p.y = a.y;
    p.out = a.out;
    p.lda = a.lda;
    p.ldy = a.ldy;
    p.ldo = a.ldo;
    p.ldm = a.Lk;
    p.q = a.q;
    p.k = a.k;
    p.mask = a.mask;
    p.mask_rows = a.mask_rows;
    p.table = a.table;
    p.table_f32 = a.table_f32;
    p.lens = a.lens;
    p.q_pos = a.q_pos;
    p.H = a.H;
    p.Lq = a.Lq;
    p.Lk = a.Lk;
    p.rows = plan.rows;
    p.chunks = plan.chunks;
    p.causal = a.causal;
    p.scale = a.scale;
    p.ea = extent(a.a, rows, a.lda);
    p.ey = extent(a.y, rows, a.ldy);
    p.em = extent(a.mask, a.mask_rows, a.Lk);
    p.part = BWD && a.dtable ? a.part : nullptr;
    p.bk = *a.buckets;
    // Distances a block can meet, or the buckets' span: whichever is less.
    const int last = p.bk.n ? p.bk.edge[p.bk.n - 1] : 1;
    const int64_t span = std::min<int64_t>((int64_t)last * (p.bk.both ? 2 : 1) + 1, (int64_t)a.Lk + plan.rows);
    const int64_t entries = span + 2 * V;
    const size_t words = (size_t)(entries + entries / V + 1) * (BWD ? (p.part ? sh.teams : 0) : 1);
    const size_t smem = words * sizeof(float);
    cudaError_t e = smem > 40 * 1024 ? allow_smem(kern, smem) : cudaSuccess;
    if (e != cudaSuccess) return e;
    void* args[] = {&p};
    e = launch_kernel(kern, dim3((unsigned)((int64_t)a.B * a.H * plan.chunks)), dim3(sh.W * sh.teams * 32), smem, stream,
                      args, false);
    if (e != cudaSuccess) return e;
    *launches = 1;
    if (p.part) {
        e = launch_rel_table(a, plan, stream);
        if (e == cudaSuccess) *launches = 2;
    }
    return e;
}

}  // namespace
}  // namespace lnk
