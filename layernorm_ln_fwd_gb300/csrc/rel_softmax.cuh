// rel_softmax.cuh -- softmax of attention scores with a learned relative position bias, and its gradients.
//
// For sequence b, head h, query i at position p = q_pos[b] + i and key j at distance d = j - p:
//   z_j = scale x_j + table[bucket(d), h] + mask_j,   y = softmax(z) over the keys that take part,
//   dS = y (dy - sum dy y),  dx = scale dS,  dtable[k, h] = sum of dS over b, i and the j of bucket k.
// A key of lens[b] or more, or behind its query where the call is causal, takes no part, and nor does one
// whose z is -inf: y = 0 there, and a row with nothing left is 0 throughout.
//
// Buckets.  Beyond the last edge every distance of a side has one bucket, so that a head needs its column of the
// table at a window of distances only (183 of them for 32 buckets up to 128), whatever the rows' length, spread
// out in shared memory.  The gradient goes the same way back: dS is added into a window by distance with loads
// and stores (a row meets each distance once), both far ends in registers, and a head's window is cut into buckets
// when the block is through with the head.  Nothing is atomic; the order of all sums is fixed by the sizes.
//
// Blocks.  A row is held in registers by 1 to 16 warps (a team), read once and written once; what a causal
// row or a short sequence leaves out is not read.  The grid is one wave of resident blocks; a block has an equal,
// contiguous share of the units (one row for each of its teams), which are ordered by head (so that a block fills
// its window once or twice), then by query from both ends inwards (a causal row's work grows with its query:
// neighbours average), then by sequence.  Its teams meet only where the head changes.
// Rows of more columns than 16 warps hold are gone through twice, in the forward by the blocks of a cluster where
// there are few of them.
#pragma once

#include <limits.h>

#include <algorithm>
#include <type_traits>
#include <utility>

#include "ckpt8.cuh"
#include "rel_ops.h"
#include "row_io.cuh"
#include "vocab.cuh"

namespace lnk {
namespace {

constexpr float kRelLog2e = 1.4426950408889634f;
constexpr int kRelMaxCluster = 8;

struct RelParams {
    const void* a;
    const void* y;
    void* out;
    unsigned lda, ldy, ldo, ldm;  // bytes between rows
    int8_t* q;
    uint8_t* k;
    const void* mask;
    unsigned mask_rows;
    const void* table;
    int table_f32;
    const int* lens;
    const int* q_pos;
    int B, H, Lq, Lk, causal;
    int dlo, dhi;        // the window's distances
    int stage;           // where the next row's values lie in the block's shared memory (backward), bytes
    int per_matrix;      // units of a sequence and head
    int64_t per_head, units;
    float scale;
    Extent ea, ey;
    float* part;
    RelBuckets bk;
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

// The distances a .. b of bucket k.
__device__ __forceinline__ void rel_distances(const RelBuckets& bk, const int* edge, int k, int& a, int& b) {
    const int side = bk.n + 1, j = k < side ? k : k - side;
    const int near = j ? edge[j - 1] : 0, far = j < bk.n ? edge[j] - 1 : INT_MAX;
    if (k < side) {
        a = far == INT_MAX ? INT_MIN : -far;
        b = j == 0 && !bk.both ? INT_MAX : -near;
    } else {
        a = max(near, 1);
        b = far;
    }
}

// The bias of head h at distance d.
__device__ __forceinline__ float rel_bias(const RelParams& p, const int* edge, int h, int d) {
    const int at = rel_bucket(p.bk, edge, d) * p.H + h;
    return p.table_f32 ? __ldg(static_cast<const float*>(p.table) + at)
                       : __bfloat162float(static_cast<const __nv_bfloat16*>(p.table)[at]);
}

// The block's units of a head, one after another: `c`-th of it is row group j (from both ends inwards)
// of sequence b.
struct RelWalk {
    int j, b;
    __device__ __forceinline__ RelWalk(const RelParams& p, int64_t c) : j((int)(c / p.B)), b((int)(c - (int64_t)j * p.B)) {}
    __device__ __forceinline__ void next(const RelParams& p) {
        if (++b == p.B) {
            b = 0;
            ++j;
        }
    }
    __device__ __forceinline__ int group(const RelParams& p) const {
        return j & 1 ? p.per_matrix - 1 - (j >> 1) : j >> 1;
    }
};

// A team's row of a unit.  Teams take the unit's rows by their positions, so that a team meets the same
// positions modulo TEAMS whatever q_pos is.
struct RelRow {
    bool ok = false;
    int n = 0;         // keys that take part: the first n columns
    int at = 0;        // the query's position
    unsigned row = 0;  // in the call
};

template <int TEAMS>
__device__ __forceinline__ RelRow rel_row(const RelParams& p, const RelWalk& w, int h, int team) {
    RelRow r;
    const int start = p.q_pos ? min(max(__ldg(p.q_pos + w.b), -kRelFar), kRelFar) : 0;
    const int len = p.lens ? min(max(__ldg(p.lens + w.b), 0), p.Lk) : p.Lk;
    const int i = w.group(p) * TEAMS + ((team - start) & (TEAMS - 1));
    r.ok = i < p.Lq;
    r.at = start + i;
    r.n = r.ok ? (p.causal ? min(len, max(r.at + 1, 0)) : len) : 0;
    r.row = (unsigned)(w.b * p.H + h) * (unsigned)p.Lq + (unsigned)i;
    return r;
}

// Row `row` of a tensor whose rows are `ld` bytes apart.
template <typename T>
__device__ __forceinline__ T* rel_at(const void* t, unsigned row, unsigned ld) {
    return reinterpret_cast<T*>(static_cast<char*>(const_cast<void*>(t)) + (unsigned long long)row * ld);
}

// Elements between the last 16-byte boundary and a row's start.
template <typename T>
__device__ __forceinline__ int rel_shift(const T* row) {
    return (int)((unsigned)reinterpret_cast<uintptr_t>(row) & 15u) / (int)sizeof(T);
}

template <int W, int TEAMS>
__device__ __forceinline__ void team_sync(int team) {
    if constexpr (TEAMS == 1)
        __syncthreads();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(W * 32) : "memory");
}

// The largest of three (one instruction of sm_100-family SMs).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// How rows lie.  kRelWhole: at multiples of 16 bytes, of whole vectors.  kRelShifted: the rows of all tensors
// start at the same place in 16 bytes, and lanes hold the aligned chunks: column c of a row that starts `sh`
// elements into a chunk is "place" c + sh, and its position p counts as p + sh, so that the distances are the
// same.  Only a row's first and last chunk are partly others'.  kRelAny: whatever else (tensors that lie differently,
// checkpoints of rows that are not of whole vectors, rows in tiles), moved into columns: two loads a vector and its
// stores put together from two lanes'.  bf16 16 x 12 x 501 x 501: 44 us shifted, 70 moved; backward 86 and 92.
constexpr int kRelAny = 0, kRelWhole = 1, kRelShifted = 2;

// Blocks an SM that the registers are to allow (rel_shape has figures; rows that are moved hold two chunks a vector).
constexpr int rel_resident(int lanes, int teams, int nv, int mode) {
    if (lanes * teams != 256) return 1;
    const int most = nv == 4 ? 3 : 4;
    return mode != kRelAny ? most : most - 1;
}

// Over groups of L lanes.
template <int L>
__device__ __forceinline__ float rel_warp_max(float a) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(kFullMask, a, o));
    return a;
}
template <int L>
__device__ __forceinline__ float rel_warp_sum(float a) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) a += __shfl_xor_sync(kFullMask, a, o);
    return a;
}

// 1 / s to one unit in the last place (s >= 1/2 but for what is infinite or NaN).
__device__ __forceinline__ float rcp_fast(float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return r;
}

// The weights of a warp (or tile) whose largest score is m are formed as exp2(z log2 e - p), p = m log2 e as rounded: the
// factor exp2(p - m log2 e) that all of them lack.  A row of one warp does without it, since it cancels; the sums of
// several warps, of which each has its own, are given it before they meet.  1 for an m that is subtracted first (`weights`).
constexpr float kRelLarge = 16777216.f;
__device__ __forceinline__ float rel_fix(float m) {
    return fabsf(m) < kRelLarge ? ex2_fast(-__fmaf_rn(m, kRelLog2e, -__fmul_rn(m, kRelLog2e))) : 1.f;
}

// exp2((m - M) log2 e), the factor from sums taken against m to those against M >= m; 1 for a sum that
// met nothing (m = -inf), which is 0, or NaN.
__device__ __forceinline__ float rel_factor(float m, float M) {
    return m == -INFINITY ? 1.f : ex2_fast((m - M) * kRelLog2e);
}

// ---------------------------------------------------------------------------------------
// The window in shared memory.
//
// Slots: for windows of up to kRelSlotBytes.  A row at position p meets distance d in column d + p, so that its
// vectors of V columns start at one residue of V throughout, and rows V positions apart at the same.  The window
// is kept SLOTS times (a row has slot p % SLOTS), each moved so that its rows' vectors are groups of V consecutive
// entries: a vector is V / 4 loads of 128 bits, one after another over the lanes, at a group held between the
// first and the last, which are the far ends' throughout.  SLOTS is 8, or TEAMS where that is more: a team's rows
// come every TEAMS positions, and TEAMS divides SLOTS, so that in the backward each slot is added to by one team
// alone.  The backward's shifted rows (below), whose residue is not their position's, have V slots for each team.
//
// Entry t of a slot stands for distance dlo + t + residue - (2 V - 1): group 0 ends before dlo whatever the
// residue, and the last group begins at dhi or behind.  The groups' first halves come first, then their second
// halves (V = 8), so that 32 lanes read 512 consecutive bytes.
//
// One window (any size; blocks of one team): entry t, for distance dlo + t - V, is at t + t / V: lanes read V
// consecutive entries each, V apart, and the spare word behind every V moves them to different banks.
// ---------------------------------------------------------------------------------------
__host__ __device__ constexpr int rel_entries(int span, int V) { return span + 2 * V; }
__host__ __device__ constexpr int rel_spread(int t, int V) { return t + (int)((unsigned)t / (unsigned)V); }

template <typename T, int SLOTS>
struct RelWindow {
    static constexpr int V = Io<T>::kVec, H = Pairs<T>::kPairs;
    float* win;
    int size;    // groups of a slot, or entries
    int dlo, dhi;

    __device__ __forceinline__ RelWindow(const RelParams& p, float* w)
        : win(w), size(SLOTS ? rel_groups(p.dhi - p.dlo + 1, V) : rel_entries(p.dhi - p.dlo + 1, V)), dlo(p.dlo), dhi(p.dhi) {}
    __device__ __forceinline__ int words() const { return SLOTS ? SLOTS * size * V : rel_spread(size - 1, V) + 1; }

    // The shift of a slot's entries, and the group (entry) of column 0 of the row at position p.
    __device__ __forceinline__ int residue(int s) const { return (2 * V - 1 - dlo - s) & (V - 1); }
    __device__ __forceinline__ int first(int p) const {
        return SLOTS ? (2 * V - 1 - dlo - p) >> (V == 8 ? 3 : 2) : V - dlo - p;
    }
    // Where entry u of slot s is.
    __device__ __forceinline__ int place(int s, int u) const {
        return s * size * V + ((u % V / 4) * size + u / V) * 4 + u % 4;
    }

    // The bias of head h; all threads, between two barriers of the caller's.
    __device__ void fill(const RelParams& p, const int* edge, int h, int threads) {
        if constexpr (SLOTS) {
            const int span = dhi - dlo + 1, per = size * V;
            float* one = win + words();
            for (int t = threadIdx.x; t < span; t += threads) one[t] = rel_bias(p, edge, h, dlo + t);
            __syncthreads();
            for (int u = threadIdx.x; u < per; u += threads)
#pragma unroll
                for (int s = 0; s < SLOTS; ++s)
                    win[place(s, u)] = one[min(max(u + residue(s) - (2 * V - 1), 0), span - 1)];
        } else {
            for (int t = threadIdx.x; t < size; t += threads)
                win[rel_spread(t, V)] = rel_bias(p, edge, h, min(max(dlo + t - V, dlo), dhi));
        }
    }
    __device__ void clear(int threads) {
        for (int t = threadIdx.x; t < words(); t += threads) win[t] = 0.f;
    }

    // -1, 0, 1: the vector of column col (vector v) lies below the window, meets it, or lies above.
    __device__ __forceinline__ int side(int first, int col) const {
        if constexpr (SLOTS) {
            const int g = first + col / V;
            return g <= 0 ? -1 : g >= size - 1 ? 1 : 0;
        } else {
            const int t = first + col;
            return t <= 1 ? -1 : t >= size - V ? 1 : 0;
        }
    }
    __device__ __forceinline__ void read(int slot, int first, int col, f2 (&b)[H]) const {
        if constexpr (SLOTS) {
            const float4* q = reinterpret_cast<const float4*>(win) + slot * size * (V / 4) +
                              min(max(first + col / V, 0), size - 1);
#pragma unroll
            for (int j = 0; j < V / 4; ++j) {
                const float4 f = q[j * size];
                b[2 * j] = f2_make(f.x, f.y);
                b[2 * j + 1] = f2_make(f.z, f.w);
            }
        } else {
            const int t = min(max(first + col, 0), size - V), c = t & (V - 1);
            const float* w = win + rel_spread(t, V);
#pragma unroll
            for (int h = 0; h < H; ++h)
                b[h] = f2_make(w[2 * h + (c + 2 * h >= V)], w[2 * h + 1 + (c + 2 * h + 1 >= V)]);
        }
    }
    // Adds a vector that meets the window.
    __device__ __forceinline__ void add(int slot, int first, int col, const f2 (&d)[H]) {
        if constexpr (SLOTS) {
            float4* q = reinterpret_cast<float4*>(win) + slot * size * (V / 4) + first + col / V;
            float4 f[V / 4];
#pragma unroll
            for (int j = 0; j < V / 4; ++j) f[j] = q[j * size];
#pragma unroll
            for (int j = 0; j < V / 4; ++j) {
                const f2 a = f2_add(f2_make(f[j].x, f[j].y), d[2 * j]);
                const f2 b = f2_add(f2_make(f[j].z, f[j].w), d[2 * j + 1]);
                q[j * size] = make_float4(f2_lo(a), f2_hi(a), f2_lo(b), f2_hi(b));
            }
        } else {
            const int t = first + col, c = t & (V - 1);
            float* w = win + rel_spread(t, V);
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
    // (one window) Into the entries beyond its ends.
    __device__ __forceinline__ void add_far(float below, float above) {
        win[0] += below;
        win[rel_spread(size - 1, V)] += above;
    }
    // What was added at distance dlo + t, at the window's ends with what is held to them.
    __device__ __forceinline__ float sum_at(int t) const {
        const int span = dhi - dlo + 1;
        float sum = 0.f;
        if constexpr (SLOTS) {
            const int last = (size - 1) * V - 1;
#pragma unroll
            for (int s = 0; s < V; ++s) {  // slots s, s + V, ... have one residue
                const int u = t + 2 * V - 1 - residue(s);
                for (int e = t == 0 ? V : max(u, V); e <= (t == span - 1 ? last : min(u, last)); ++e) {
                    const float* w = win + place(s, e);
#pragma unroll
                    for (int k = 0; k < SLOTS / V; ++k) sum += w[k * V * V * size];
                }
            }
        } else {
            for (int e = t == 0 ? 0 : t + V; e <= (t == span - 1 ? size - 1 : t + V); ++e) sum += win[rel_spread(e, V)];
        }
        return sum;
    }
};

// ---------------------------------------------------------------------------------------
// Forward.
// ---------------------------------------------------------------------------------------

// LPR lanes (of 1 to 16 warps, or a part of one) hold a row, NV vectors each (lane l: vectors l, l + LPR, ...);
// TEAMS rows at a time.  The next row's loads are under way during the current one's arithmetic, but for kRelAny.
// LOOP: rows of any length, in tiles of that size, twice.
//
// One read of the scores, one write of the probabilities: bf16 16 x 12 x 512 x 512 with lengths 34.4 us, 0.81 of the
// measured copy rate; in full 0.86.  What is left is issue: a vector is unpacked, given its bias (two 128-bit shared loads),
// 8 exponents, and packed.  A decode step (bf16 64 x 16 x 1 x 4096 with lengths) takes 6.9 us for 2.3 of traffic: a launch,
// and a row's time from its first load to its last store.
template <typename T, int LPR, int TEAMS, int NV, bool LOOP, bool CKPT, int MODE, bool SLOTS>
__global__ void __launch_bounds__(LPR* TEAMS, rel_resident(LPR, TEAMS, NV, MODE)) rel_fwd_kernel(const __grid_constant__ RelParams p) {
    constexpr int V = Io<T>::kVec, H = Pairs<T>::kPairs;
    constexpr int W = LPR > 32 ? LPR / 32 : 1, L = LPR > 32 ? 32 : LPR;  // warps of a row, its lanes in a warp
    constexpr int kThreads = LPR * TEAMS;
    constexpr int kTile = LPR * NV * V, kPiece = L * V;
    constexpr bool SHIFT = MODE == kRelShifted, AHEAD = MODE != kRelAny;
    static_assert(SLOTS || TEAMS == 1, "one window has one team");
    static_assert(!SHIFT || (SLOTS && !CKPT), "shifted rows start in 16 bytes where they do");
    extern __shared__ __align__(16) float smem[];
    __shared__ int edge[kRelMaxEdges];
    __shared__ float red[2][TEAMS][2][W];
    __shared__ float2 joint[2][LOOP ? kRelMaxCluster : 1];  // the cluster's (max, sum)
    const int cluster = LOOP ? (int)cluster_blocks() : 1, rank = LOOP ? (int)cluster_rank() : 0;
    if (cluster > 1) cluster_arrive();  // "this block's shared memory exists"
    const int tid = threadIdx.x, lane = tid & (L - 1);
    const int team = tid / LPR, wt = W == 1 ? 0 : (tid - team * LPR) / 32;
    for (int i = tid; i < p.bk.n; i += kThreads) edge[i] = p.bk.edge[i];
    pdl_enter();
    constexpr int kSlots = SLOTS ? rel_slot_count(TEAMS) : 0;
    RelWindow<T, kSlots> win(p, smem);
    const f2 scale = f2_splat(p.scale), l2 = f2_splat(kRelLog2e);
    // A warp's k-th piece of a row, in vectors.  Where vectors are moved into columns a warp's pieces follow one
    // another, so that it stores the chunks between them whole; else the row's warps take turns.
    auto place_of = [&](int k) { return MODE == kRelAny ? (wt * NV + k) * L : k * LPR + wt * 32; };
    const int blocks = ckpt_blocks(p.Lk);
    const unsigned block = blockIdx.x / cluster, grid = gridDim.x / cluster;
    const int64_t end = p.units * ((int64_t)block + 1) / grid;
    int parity = 0;
    if (cluster > 1) cluster_wait();
    for (int64_t unit = p.units * block / grid; unit < end;) {
        const int h = (int)(unit / p.per_head);
        const int64_t c0 = unit - (int64_t)h * p.per_head;
        const int count = (int)(min(p.per_head, c0 + (end - unit)) - c0);
        unit += count;
        __syncthreads();
        win.fill(p, edge, h, kThreads);
        __syncthreads();
        uint4 raw[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) raw[k] = make_uint4(0, 0, 0, 0);
        // (shifted rows)
        auto chunk = [&](const RelRow& r, const T* x, int sh) {
            const T* mine = x + ((wt * 32 + lane) * V - sh);
            const int n = r.n > 0 ? sh + r.n - (wt * 32 + lane) * V : 0;
            return [=](int k, const char*& c) {
                c = reinterpret_cast<const char*>(mine + k * LPR * V);
                return k * LPR * V < n;
            };
        };
        auto load = [&](const RelRow& r, int base) {
            const T* x = rel_at<const T>(p.a, r.row, p.lda);
            const RowIn<T> in(x, p.Lk, p.ea);
            const int sh = SHIFT ? rel_shift(x) : 0;
            auto column = [&](int k) { return base + (place_of(k) + lane) * V; };
            if constexpr (MODE == kRelWhole) {
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    if (column(k) < r.n) raw[k] = __ldcs(reinterpret_cast<const uint4*>(x + column(k)));
            } else if constexpr (SHIFT) {
                load_chunks<T>(raw, in.inside, chunk(r, x, sh));
            } else {
                load_vectors<T>(raw, in, r.n, p.ea, column);
            }
        };
        RelWalk walk(p, c0);
        RelRow r = rel_row<TEAMS>(p, walk, h, team);
        if (!LOOP) load(r, 0);
        for (int c = 0; c < count; ++c) {
            f2 z[NV][H];
            const int sh = SHIFT ? rel_shift(rel_at<const T>(p.a, r.row, p.lda)) : 0;
            const int n = sh + r.n, at = r.at + sh, first = win.first(at), slot = at & (kSlots - 1);
            const int most = L < 32 ? __reduce_max_sync(kFullMask, n) : n;   // of the warp's rows
            const int least = L < 32 ? __reduce_min_sync(kFullMask, n) : n;
            const unsigned row = r.row;
            const bool ok = r.ok;
            const T* mrow = p.mask ? rel_at<const T>(p.mask, row % p.mask_rows, p.ldm) : nullptr;
            if constexpr (SHIFT) {
                const T* x = rel_at<const T>(p.a, row, p.lda);
                end_chunks<T>(raw, RowIn<T>(x, p.Lk, p.ea).inside, p.ea, chunk(r, x, sh));
            }
            // The scores of a tile, where the warp's 32 vectors have keys that take part (elsewhere z is
            // left as it is, and not used): -inf at the others among them.  Returns the largest.
            auto scores = [&](int base) {
                float m = -INFINITY;
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int from = base + place_of(k) * V, col = from + lane * V;
                    if (from >= most) continue;
                    f2 b[H];
                    win.read(slot, first, col, b);
                    Pairs<T>::unpack(raw[k], z[k]);
#pragma unroll
                    for (int h2 = 0; h2 < H; ++h2) z[k][h2] = f2_fma(scale, z[k][h2], b[h2]);
                }
                if (mrow) {
#pragma unroll
                    for (int k = 0; k < NV; ++k) {
                        const int col = base + (place_of(k) + lane) * V;
                        if (col >= n) continue;
                        f2 mv[H];
                        if constexpr (MODE == kRelWhole) {
                            Pairs<T>::unpack(ld_keep(mrow + col), mv);
                        } else {  // element by element: few registers, and a mask is small and read again
#pragma unroll
                            for (int h2 = 0; h2 < H; ++h2) {
                                const int c = col - sh + 2 * h2;
                                mv[h2] = f2_make(c >= 0 && c < n - sh ? Io<T>::to_f(mrow[c]) : 0.f,
                                                 c >= -1 && c + 1 < n - sh ? Io<T>::to_f(mrow[c + 1]) : 0.f);
                            }
                        }
#pragma unroll
                        for (int h2 = 0; h2 < H; ++h2) {  // a mask of -inf removes a key whatever its score is
                            const f2 s = f2_add(z[k][h2], mv[h2]);
                            z[k][h2] = f2_make(f2_lo(mv[h2]) == -INFINITY ? -INFINITY : f2_lo(s),
                                               f2_hi(mv[h2]) == -INFINITY ? -INFINITY : f2_hi(s));
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int from = base + place_of(k) * V, col = from + lane * V;
                    if (from >= most) continue;
                    if (from + kPiece > least) {
                        const int left = n - col;
#pragma unroll
                        for (int h2 = 0; h2 < H; ++h2)
                            z[k][h2] = f2_make(2 * h2 < left ? f2_lo(z[k][h2]) : -INFINITY,
                                               2 * h2 + 1 < left ? f2_hi(z[k][h2]) : -INFINITY);
                    }
                    if (SHIFT && from == 0) {
#pragma unroll
                        for (int h2 = 0; h2 < H; ++h2)
                            z[k][h2] = f2_make(col + 2 * h2 >= sh ? f2_lo(z[k][h2]) : -INFINITY,
                                               col + 2 * h2 + 1 >= sh ? f2_hi(z[k][h2]) : -INFINITY);
                    }
#pragma unroll
                    for (int h2 = 0; h2 < H; ++h2) m = max3(m, f2_lo(z[k][h2]), f2_hi(z[k][h2]));
                }
                return m;
            };
            // z becomes exp(z - m), but for the factor rel_fix(m); returns its sum.  exp2(z log2 e - m log2 e): the last
            // product's rounding is the same for the whole warp.  For an m whose rounding could pass fp32's exponents,
            // z - m first.
            auto weights = [&](float m, int base) {
                float ref = m == -INFINITY ? 0.f : m;
                if (!(fabsf(ref) < kRelLarge)) {
#pragma unroll
                    for (int k = 0; k < NV; ++k) {
                        if (base + place_of(k) * V >= most) continue;
#pragma unroll
                        for (int h2 = 0; h2 < H; ++h2) z[k][h2] = f2_add(z[k][h2], f2_splat(-ref));
                    }
                    ref = 0.f;
                }
                const f2 nr = f2_splat(__fmul_rn(-ref, kRelLog2e));
                f2 acc = f2_splat(0.f);
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    if (base + place_of(k) * V >= most) continue;
#pragma unroll
                    for (int h2 = 0; h2 < H; ++h2) {
                        const f2 t = f2_fma(z[k][h2], l2, nr);
                        z[k][h2] = f2_make(ex2_fast(f2_lo(t)), ex2_fast(f2_hi(t)));
                        acc = f2_add(acc, z[k][h2]);
                    }
                }
                return f2_lo(acc) + f2_hi(acc);
            };
            float m = -INFINITY, s = 0.f;
            if constexpr (LOOP) {
                for (int base = rank * kTile; base < n; base += cluster * kTile) {
                    load(r, base);
                    const float mt = fmaxf(m, rel_warp_max<L>(scores(base)));
                    s *= rel_factor(m, mt);
                    m = mt;
                    s += weights(m, base) * rel_fix(m);
                }
            } else {
                m = scores(0);
                walk.next(p);
                r = c + 1 < count ? rel_row<TEAMS>(p, walk, h, team) : RelRow();
                if (AHEAD) load(r, 0);
                if (L == 32 && !ok) {  // (the same in the whole team)
                    if (!AHEAD) load(r, 0);
                    continue;
                }
                m = rel_warp_max<L>(m);
                s = weights(m, 0);
            }
            s = rel_warp_sum<L>(s);
            float inv;
            if constexpr (W == 1) {
                inv = s == 0.f ? 0.f : rcp_fast(s);
            } else {  // the warps' (max, sum) meet once
                const float fix = rel_fix(m);
                if (lane == 0) {
                    red[parity][team][0][wt] = m;
                    red[parity][team][1][wt] = LOOP ? s : s * fix;
                }
                team_sync<W, TEAMS>(team);
                float M = -INFINITY, S = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w) M = fmaxf(M, red[parity][team][0][w]);
#pragma unroll
                for (int w = 0; w < W; ++w) S += red[parity][team][1][w] * rel_factor(red[parity][team][0][w], M);
                if (LOOP && cluster > 1) {  // and the blocks'
                    if (tid < cluster) {
                        const uint32_t to = in_block(&joint[parity][rank], (uint32_t)tid);
                        st_cluster_f32(to, M);
                        st_cluster_f32(to + 4, S);
                    }
                    cluster_arrive();
                    cluster_wait();
                    M = -INFINITY;
                    S = 0.f;
                    for (int i = 0; i < cluster; ++i) M = fmaxf(M, joint[parity][i].x);
                    for (int i = 0; i < cluster; ++i) S += joint[parity][i].y * rel_factor(joint[parity][i].x, M);
                }
                inv = S == 0.f ? 0.f : fix * rel_factor(m, M) / S;
                parity ^= 1;
            }
            const f2 c2 = f2_splat(inv);
            T* y = rel_at<T>(p.out, row, p.ldo);
            const int stored = L == 32 || ok ? sh + p.Lk : 0;
            // The warp's last place: rows that share a warp start at different places of a chunk, and all lanes take
            // part in a piece's stores.
            const int reach = SHIFT && L < 32 ? __reduce_max_sync(kFullMask, sh + p.Lk) : sh + p.Lk;
            for (int base = LOOP ? rank * kTile : 0; base < (LOOP ? p.Lk : 1); base += cluster * kTile) {
                RowOut<T, L> out;
                if constexpr (LOOP) {
                    load(r, base);
                    scores(base);
                    weights(m, base);
                }
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int from = base + place_of(k) * V, col = from + lane * V;
                    if (from >= reach) continue;
                    uint4 u = make_uint4(0, 0, 0, 0);
                    if (from < most) {
#pragma unroll
                        for (int h2 = 0; h2 < H; ++h2) z[k][h2] = f2_mul(z[k][h2], c2);
                        u = Pairs<T>::pack(z[k]);
                        if (inv != inv) u = first_of<T>(u, n - col);  // (0 times NaN)
                    }
                    if constexpr (MODE == kRelWhole) {
                        if (col < stored) st_stream(y + col, u);
                    } else if constexpr (SHIFT) {
                        store_chunks<T, L>(y + (col - sh), from, sh, stored, u);
                    } else {
                        out.put(y, col, stored, u, k == 0, k == NV - 1);
                    }
                    if constexpr (CKPT)
                        ckpt_keep<T>(u, col, L == 32 || ok ? blocks * kCkptBlock : 0, p.q + (unsigned long long)row * (blocks * kCkptBlock),
                                     p.k + (unsigned long long)row * blocks);
                }
            }
            if constexpr (LOOP) {
                walk.next(p);
                if (c + 1 < count) r = rel_row<TEAMS>(p, walk, h, team);
            } else if (!AHEAD) {
                load(r, 0);
            }
        }
    }
}

// ---------------------------------------------------------------------------------------
// Backward.
// ---------------------------------------------------------------------------------------

// A vector times a power of two.
template <typename T>
__device__ __forceinline__ uint4 rel_times(const uint4& u, float f) {
    f2 v[Pairs<T>::kPairs];
    Pairs<T>::unpack(u, v);
#pragma unroll
    for (int h = 0; h < Pairs<T>::kPairs; ++h) v[h] = f2_mul(v[h], f2_splat(f));
    return Pairs<T>::pack(v);
}

// A row's probabilities: stored in T, or in 8 bits.
template <typename T, bool CKPT>
struct Probs {
    uint4 u;
    __device__ __forceinline__ void clear() { u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void first(int count) { u = first_of<T>(u, count); }
    __device__ __forceinline__ void values(f2 (&v)[Pairs<T>::kPairs]) const { Pairs<T>::unpack(u, v); }
    __device__ __forceinline__ void twice() { u = rel_times<T>(u, 2.f); }
};
template <typename T>
struct Probs<T, true> {
    CkptRaw<T> r;
    __device__ __forceinline__ void clear() { r.clear(); }
    __device__ __forceinline__ void first(int count) { r.first(count); }
    __device__ __forceinline__ void values(f2 (&v)[Pairs<T>::kPairs]) const { r.values(v); }
    __device__ __forceinline__ void twice() { r.k += r.k - 1u < 253u; }  // (the step; 0 and 255 have none)
};

// 0 where y is, whatever g is.
__device__ __forceinline__ f2 where_weight(f2 y, f2 g) {
    return f2_make(f2_lo(y) == 0.f ? 0.f : f2_lo(g), f2_hi(y) == 0.f ? 0.f : f2_hi(g));
}

// As the forward's.  The next row's dy and y lie in shared memory by the time they are wanted, each lane's copied
// by itself (cp.async: no registers hold them meanwhile, and no barrier is needed), for rows of whole vectors: bf16
// 12 x 4096 x 4096 189 us, 235 by loads in time; 16 x 12 x 512 x 512 57 and 126.  Shifted rows measured slower so (the
// end chunks of their two tensors go by other loads, between the copies) and load in time.  bf16 16 x 12 x 512 x 512
// with lengths and the table's gradient 54.5 us, 0.75 of the measured copy rate; what is left is issue (the window's load,
// add and store for the vectors that meet it, and integers to fp32 from a checkpoint).
template <typename T, int LPR, int TEAMS, int NV, bool LOOP, bool CKPT, int MODE, bool SLOTS>
__global__ void __launch_bounds__(LPR* TEAMS, rel_resident(LPR, TEAMS, NV, MODE)) rel_bwd_kernel(const __grid_constant__ RelParams p) {
    constexpr int V = Io<T>::kVec, H = Pairs<T>::kPairs;
    constexpr int W = LPR > 32 ? LPR / 32 : 1, L = LPR > 32 ? 32 : LPR;  // warps of a row, its lanes in a warp
    constexpr int kThreads = LPR * TEAMS, kWarps = kThreads / 32;
    constexpr int kTile = LPR * NV * V, kPiece = L * V;
    constexpr bool SHIFT = MODE == kRelShifted;
    static_assert(SLOTS || TEAMS == 1, "one window has one team");
    static_assert(!SHIFT || (SLOTS && !CKPT && L == 32), "shifted rows start in 16 bytes where they do");
    extern __shared__ __align__(16) float smem[];
    __shared__ int edge[kRelMaxEdges];
    __shared__ float red[2][TEAMS][W];
    __shared__ float far_sums[kWarps][2];
    const int tid = threadIdx.x, lane = tid & (L - 1), warp = tid >> 5;
    const int team = tid / LPR, wt = W == 1 ? 0 : (tid - team * LPR) / 32;
    for (int i = tid; i < p.bk.n; i += kThreads) edge[i] = p.bk.edge[i];
    pdl_enter();
    // Shifted rows' residues follow their rows, not their positions: a team has slots of its own.
    constexpr int kSlots = !SLOTS ? 0 : SHIFT ? TEAMS * V : rel_slot_count(TEAMS);
    RelWindow<T, kSlots> win(p, smem);
    const bool sums = p.part != nullptr;
    // The next row's dy and y (or integers), copied by each lane for itself while it works on the current one.
    constexpr bool STAGED = MODE == kRelWhole;
    constexpr int kBytes = CKPT ? V : 16;
    unsigned char* stage_dy = reinterpret_cast<unsigned char*>(smem) + p.stage + tid * 16;
    unsigned char* stage_y = reinterpret_cast<unsigned char*>(smem) + p.stage + NV * kThreads * 16 + tid * kBytes;
    const f2 scale = f2_splat(p.scale);
    // A warp's k-th piece of a row, in vectors.  Where vectors are moved into columns a warp's pieces follow one
    // another, so that it stores the chunks between them whole; else the row's warps take turns.
    auto place_of = [&](int k) { return MODE == kRelAny ? (wt * NV + k) * L : k * LPR + wt * 32; };
    const int blocks = ckpt_blocks(p.Lk);
    const int64_t end = p.units * ((int64_t)blockIdx.x + 1) / gridDim.x;
    int parity = 0;
    for (int64_t unit = p.units * blockIdx.x / gridDim.x; unit < end;) {
        const int h = (int)(unit / p.per_head);
        const int64_t c0 = unit - (int64_t)h * p.per_head;
        const int count = (int)(min(p.per_head, c0 + (end - unit)) - c0);
        unit += count;
        if (sums) {
            __syncthreads();
            win.clear(kThreads);
            __syncthreads();
        }
        f2 below = f2_splat(0.f), above = f2_splat(0.f);  // dS of the far ends
        uint4 g[NV];
        Probs<T, CKPT> pr[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            g[k] = make_uint4(0, 0, 0, 0);
            pr[k].clear();
        }
        RelWalk walk(p, c0);
        uint32_t kn[CKPT ? NV : 1];
        auto issue = [&](const RelRow& r) {
            const T* dy = rel_at<const T>(p.a, r.row, p.lda);
            const T* py = rel_at<const T>(p.y, r.row, p.ldy);
            const int8_t* pq = p.q + (unsigned long long)r.row * (blocks * kCkptBlock);
            const uint8_t* pk = p.k + (unsigned long long)r.row * blocks;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int col = (place_of(k) + lane) * V;
                if (col < r.n) {
                    copy_async<16>(stage_dy + k * (kThreads * 16), dy + col);
                    if constexpr (CKPT) {
                        copy_async<V>(stage_y + k * (kThreads * V), pq + col);
                        kn[k] = load_ahead(pk + col / kCkptBlock);
                    } else {
                        copy_async<16>(stage_y + k * (kThreads * 16), py + col);
                    }
                }
            }
            copies_commit();
        };
        RelRow ahead = rel_row<TEAMS>(p, walk, h, team);
        if constexpr (STAGED) issue(ahead);
        for (int c = 0; c < count; ++c) {
            const RelRow r = ahead;
            walk.next(p);
            ahead = c + 1 < count ? rel_row<TEAMS>(p, walk, h, team) : RelRow();
            if (L == 32 && !r.ok) {  // (the same in the whole team)
                if constexpr (STAGED) issue(ahead);
                continue;
            }
            const T* dy = rel_at<const T>(p.a, r.row, p.lda);
            const int sh = SHIFT ? rel_shift(dy) : 0;
            const int n = sh + r.n, at = r.at + sh, first = win.first(at);
            const int slot = SHIFT ? team * V + (at & (V - 1)) : at & (kSlots - 1);
            const int most = L < 32 ? __reduce_max_sync(kFullMask, n) : n;   // of the warp's rows
            const int least = L < 32 ? __reduce_min_sync(kFullMask, n) : n;
            const int stored = L == 32 || r.ok ? sh + p.Lk : 0;
            const T* py = rel_at<const T>(p.y, r.row, p.ldy);
            const int8_t* pq = p.q + (unsigned long long)r.row * (blocks * kCkptBlock);
            const uint8_t* pk = p.k + (unsigned long long)r.row * blocks;
            T* dx = rel_at<T>(p.out, r.row, p.ldo);
            auto load = [&](int base) {
                if constexpr (STAGED) {
                    copies_wait<0>();
#pragma unroll
                    for (int k = 0; k < NV; ++k) {
                        g[k] = *reinterpret_cast<const uint4*>(stage_dy + k * (kThreads * 16));
                        if constexpr (CKPT) {
                            pr[k].r.take(stage_y + k * (kThreads * V));
                            pr[k].r.k = kn[k];
                        } else {
                            pr[k].u = *reinterpret_cast<const uint4*>(stage_y + k * (kThreads * 16));
                        }
                    }
                } else {
                    const RowIn<T> in(dy, p.Lk, p.ea), iy(py, p.Lk, p.ey);
                    auto column = [&](int k) { return base + (place_of(k) + lane) * V; };
                    auto chunk = [&](const T* row) {
                        const T* mine = row + ((wt * 32 + lane) * V - sh);
                        const int left = n > sh ? n - (wt * 32 + lane) * V : 0;
                        return [=](int k, const char*& c) {
                            c = reinterpret_cast<const char*>(mine + k * LPR * V);
                            return k * LPR * V < left;
                        };
                    };
                    uint4 y[NV];
#pragma unroll
                    for (int k = 0; k < NV; ++k) y[k] = make_uint4(0, 0, 0, 0);
                    if constexpr (SHIFT) {
                        load_chunks<T>(g, in.inside, chunk(dy));
                        load_chunks<T>(y, iy.inside, chunk(py));
                        end_chunks<T>(g, in.inside, p.ea, chunk(dy));
                        end_chunks<T>(y, iy.inside, p.ey, chunk(py));
                    } else {
                        load_vectors<T>(g, in, n, p.ea, column);
                        if constexpr (!CKPT) load_vectors<T>(y, iy, n, p.ey, column);
                    }
#pragma unroll
                    for (int k = 0; k < NV; ++k) {
                        if constexpr (!CKPT)
                            pr[k].u = y[k];
                        else if (column(k) < n)
                            pr[k].r.load(pq, pk, column(k));
                    }
                }
#pragma unroll
                for (int k = 0; k < NV; ++k) {  // zeros where a key takes no part
                    const int from = base + place_of(k) * V;
                    if (from < most && from + kPiece > least) {
                        g[k] = first_of<T>(g[k], n - from - lane * V);
                        pr[k].first(n - from - lane * V);
                    }
                    if constexpr (SHIFT) {
                        if (from == 0) {
                            g[k] = behind<T>(g[k], sh - lane * V);
                            pr[k].u = behind<T>(pr[k].u, sh - lane * V);
                        }
                    }
                }
            };
            // sum dy y over the row; `careful`: without what a weight of 0 meets.
            auto row_sum = [&](auto careful) {
                float s = 0.f;
                for (int base = 0; base < (LOOP ? n : 1); base += kTile) {
                    if constexpr (LOOP) load(base);
                    f2 acc = f2_splat(0.f);
#pragma unroll
                    for (int k = 0; k < NV; ++k) {
                        if (base + place_of(k) * V >= most) continue;
                        f2 d[H], y[H];
                        Pairs<T>::unpack(g[k], d);
                        pr[k].values(y);
#pragma unroll
                        for (int h2 = 0; h2 < H; ++h2)
                            acc = f2_fma(decltype(careful)::value ? where_weight(y[h2], d[h2]) : d[h2], y[h2], acc);
                    }
                    s += f2_lo(acc) + f2_hi(acc);
                }
                s = rel_warp_sum<L>(s);
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
            // not count) is formed again without such keys.  From 2^103 on its difference from a finite dy may pass fp32's
            // range: twice y and halves of dy and of the sum take their places.
            constexpr float kFar = 0x1p103f;
            const bool careful = L < 32 ? __any_sync(kFullMask, !(fabsf(s) < kFar)) : !(fabsf(s) < kFar);
            bool far = false;
            auto halve = [&] {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    g[k] = rel_times<T>(g[k], 0.5f);
                    pr[k].twice();
                }
            };
            if (careful) {
                s = row_sum(std::true_type{});
                far = !(fabsf(s) < kFar);
                if (far) s *= 0.5f;
                if (!LOOP && far) halve();
            }
            if constexpr (STAGED) issue(ahead);  // (what was there has been used)
            const f2 s2 = f2_splat(s);
            for (int base = 0; base < (LOOP ? p.Lk : 1); base += kTile) {
                RowOut<T, L> out;
                if constexpr (LOOP) load(base);
                if (LOOP && far) halve();
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int from = base + place_of(k) * V, col = from + lane * V;
                    if (from >= sh + p.Lk) continue;
                    uint4 u = make_uint4(0, 0, 0, 0);
                    if (from < most) {
                        f2 d[H], y[H], o[H];
                        Pairs<T>::unpack(g[k], d);
                        pr[k].values(y);
#pragma unroll
                        for (int h2 = 0; h2 < H; ++h2) d[h2] = f2_mul(y[h2], f2_sub(d[h2], s2));
                        if (careful) {
#pragma unroll
                            for (int h2 = 0; h2 < H; ++h2) {
                                d[h2] = where_weight(y[h2], d[h2]);
                                d[h2] = f2_make(col + 2 * h2 < n ? f2_lo(d[h2]) : 0.f,
                                                col + 2 * h2 + 1 < n ? f2_hi(d[h2]) : 0.f);
                                // (before a shifted row's start y is 0)
                            }
                        }
#pragma unroll
                        for (int h2 = 0; h2 < H; ++h2) o[h2] = f2_mul(scale, d[h2]);
                        u = Pairs<T>::pack(o);
                        if (sums) {
                            const int side = win.side(first, col);
                            if (side == 0) {
                                win.add(slot, first, col, d);
                            } else {
                                f2 sum = f2_add(d[0], d[1]);
#pragma unroll
                                for (int h2 = 2; h2 < H; ++h2) sum = f2_add(sum, d[h2]);
                                if (side < 0)
                                    below = f2_add(below, sum);
                                else
                                    above = f2_add(above, sum);
                            }
                        }
                    }
                    if constexpr (MODE == kRelWhole) {
                        if (col < stored) st_stream(dx + col, u);
                    } else if constexpr (SHIFT) {
                        store_chunks<T, L>(dx + (col - sh), from, sh, stored, u);
                    } else {
                        out.put(dx, col, stored, u, k == 0, k == NV - 1);
                    }
                }
            }
            if constexpr (W == 1) __syncwarp();  // the next row's entries are other lanes'
        }
        if (!sums) continue;
        // The head is through with: its window by distance, then by bucket.
        const float fb = rel_warp_sum<32>(f2_lo(below) + f2_hi(below)), fa = rel_warp_sum<32>(f2_lo(above) + f2_hi(above));
        if ((tid & 31) == 0) {
            far_sums[warp][0] = fb;
            far_sums[warp][1] = fa;
        }
        __syncthreads();
        const int span = p.dhi - p.dlo + 1;
        float* one = smem + win.words();  // slots: their sum by distance
        if constexpr (SLOTS) {
            for (int t = tid; t < span; t += kThreads) {
                float v = win.sum_at(t);
                if (t == 0)
                    for (int w = 0; w < kWarps; ++w) v += far_sums[w][0];
                if (t == span - 1)
                    for (int w = 0; w < kWarps; ++w) v += far_sums[w][1];
                one[t] = v;
            }
        } else if (tid == 0) {
            for (int w = 0; w < kWarps; ++w) win.add_far(far_sums[w][0], far_sums[w][1]);
        }
        __syncthreads();
        const int total = (p.bk.n + 1) * (p.bk.both ? 2 : 1);
        float* part = p.part + ((int64_t)blockIdx.x + h) * total;
        for (int k0 = 0; k0 < total; k0 += kThreads / 4) {  // four lanes a bucket
            const int k = k0 + tid / 4;
            float v = 0.f;
            if (k < total) {
                int a, b;
                rel_distances(p.bk, edge, k, a, b);
                // (distances beyond the window have been added to its ends)
                if (a < p.dlo && b >= p.dlo) a = p.dlo;
                if (b > p.dhi && a <= p.dhi) b = p.dhi;
                if (a >= p.dlo && b <= p.dhi)
                    for (int d = a + (tid & 3); d <= b; d += 4) v += SLOTS ? one[d - p.dlo] : win.sum_at(d - p.dlo);
            }
            v += __shfl_xor_sync(kFullMask, v, 1);
            v += __shfl_xor_sync(kFullMask, v, 2);
            if (k < total && (tid & 3) == 0) part[k] = v;
        }
    }
}

// ---------------------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------------------
template <typename T, bool BWD, bool CKPT, int MODE, bool SLOTS, int I>
const void* rel_kernel_of() {
    constexpr RelShape s = kRelShapes[I];
    // Rows in tiles have one window, and one window blocks of a team of several warps; the backward's shifted rows have a
    // warp at least, and in bf16 more than 32 vectors.
    constexpr bool shifted_back = BWD && MODE == kRelShifted;
    if constexpr ((SLOTS && s.loop) || (!SLOTS && (s.teams > 1 || s.lanes == 32)) || (shifted_back && s.lanes < 32) ||
                  (shifted_back && Io<T>::kVec == 8 && s.lanes * s.nv <= 32))
        return nullptr;
    else if constexpr (BWD)
        return (const void*)rel_bwd_kernel<T, s.lanes, s.teams, s.nv, s.loop, CKPT, MODE, SLOTS>;
    else
        return (const void*)rel_fwd_kernel<T, s.lanes, s.teams, s.nv, s.loop, CKPT, MODE, SLOTS>;
}

template <typename T, bool BWD, bool CKPT, int MODE, bool SLOTS, int... I>
const void* rel_kernel(int shape, std::integer_sequence<int, I...>) {
    const void* found = nullptr;
    ((void)(shape == I && (found = rel_kernel_of<T, BWD, CKPT, MODE, SLOTS, I>())), ...);
    return found;
}

template <typename T, bool BWD>
const void* rel_kernel(int shape, bool ckpt, int mode, bool slots) {
    constexpr auto all = std::make_integer_sequence<int, kRelShapeCount>();
    if (mode == kRelShifted) return rel_kernel<T, BWD, false, kRelShifted, true>(shape, all);
    if (ckpt)
        return !slots               ? rel_kernel<T, BWD, true, kRelAny, false>(shape, all)
               : mode == kRelWhole ? rel_kernel<T, BWD, true, kRelWhole, true>(shape, all)
                                   : rel_kernel<T, BWD, true, kRelAny, true>(shape, all);
    return !slots               ? rel_kernel<T, BWD, false, kRelAny, false>(shape, all)
           : mode == kRelWhole ? rel_kernel<T, BWD, false, kRelWhole, true>(shape, all)
                               : rel_kernel<T, BWD, false, kRelAny, true>(shape, all);
}

// Whether rows of n elements, ld apart, are whole vectors at vectors' distance.
template <typename T>
bool rel_whole(const void* t, int64_t ld, int64_t n) {
    return !t || ((reinterpret_cast<uintptr_t>(t) & 15u) == 0 && ld % Io<T>::kVec == 0 && n % Io<T>::kVec == 0);
}

// Whether rows of both start at the same place in 16 bytes, every one of them.
template <typename T>
bool rel_congruent(const void* a, int64_t lda, const void* b, int64_t ldb) {
    return ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) & 15u) == 0 &&
           (lda - ldb) * (int64_t)sizeof(T) % 16 == 0;
}

template <typename T, bool BWD>
cudaError_t launch_rel_t(const RelArgs& a, cudaStream_t stream, int* launches) {
    constexpr int V = Io<T>::kVec;
    *launches = 0;
    RelParams p;
    const int64_t rows = (int64_t)a.B * a.H * a.Lq;
    auto extent = [&](const void* t, int64_t n, int64_t ld) {
        const char* c = static_cast<const char*>(t);
        return Extent{c, c ? c + ((n - 1) * ld + a.Lk) * (int64_t)sizeof(T) : c};
    };
    p.a = a.a;
    p.y = a.y;
    p.out = a.out;
    p.lda = (unsigned)(a.lda * (int64_t)sizeof(T));
    p.ldy = (unsigned)(a.ldy * (int64_t)sizeof(T));
    p.ldo = (unsigned)(a.ldo * (int64_t)sizeof(T));
    p.ldm = (unsigned)(a.Lk * sizeof(T));
    p.q = a.q;
    p.k = a.k;
    p.mask = a.mask;
    p.mask_rows = (unsigned)a.mask_rows;
    p.table = a.table;
    p.table_f32 = a.table_f32;
    p.lens = a.lens;
    p.q_pos = a.q_pos;
    p.B = a.B;
    p.H = a.H;
    p.Lq = a.Lq;
    p.Lk = a.Lk;
    p.causal = a.causal;
    p.scale = a.scale;
    p.ea = extent(a.a, rows, a.lda);
    p.ey = extent(a.y, rows, a.ldy);
    p.part = BWD && a.dtable ? a.part : nullptr;
    p.bk = *a.buckets;
    rel_span(a, &p.dlo, &p.dhi);
    const int span = p.dhi - p.dlo + 1;
    const bool whole = rel_whole<T>(a.a, a.lda, a.Lk) && rel_whole<T>(a.y, a.ldy, a.Lk) &&
                       rel_whole<T>(a.out, a.ldo, a.Lk) && rel_whole<T>(a.mask, a.Lk, a.Lk);
    bool slots;
    int mode = whole ? kRelWhole : kRelAny;
    int shape = rel_shape(V, rows, a.Lq, a.Lk, span, BWD, a.causal, &slots);
    int copies = rel_slot_count(kRelShapes[shape].teams);
    if (!whole && !a.q && slots && rel_congruent<T>(a.a, a.lda, a.out, a.ldo) &&
        (!a.y || rel_congruent<T>(a.a, a.lda, a.y, a.ldy))) {
        int shifted_copies;
        const int shifted = rel_shape_shifted(V, rows, a.Lq, a.Lk, span, BWD, &shifted_copies);
        if (shifted >= 0) {
            mode = kRelShifted;
            shape = shifted;
            copies = shifted_copies;
        }
    }
    const RelShape& sh = kRelShapes[shape];
    p.per_matrix = (a.Lq + sh.teams - 1) / sh.teams;
    p.per_head = (int64_t)p.per_matrix * a.B;
    p.units = p.per_head * a.H;
    // The forward's one copy by distance (slots), and the backward's sums by distance.
    const size_t words = BWD && !p.part ? 0
                         : slots        ? (size_t)copies * rel_groups(span, V) * V + span
                                        : (size_t)rel_spread(rel_entries(span, V) - 1, V) + 1;
    const int threads = sh.lanes * sh.teams;
    size_t smem = words * sizeof(float);
    p.stage = (int)((smem + 15) / 16 * 16);
    if (BWD && mode == kRelWhole && slots) smem = p.stage + (size_t)sh.nv * threads * (16 + (a.q ? V : 16));
    const bool ckpt = a.q != nullptr;
    const void* kern = rel_kernel<T, BWD>(shape, ckpt, mode, slots);
    if (!kern) return cudaErrorInvalidValue;
    cudaError_t e = smem > 40 * 1024 ? allow_smem(kern, smem) : cudaSuccess;
    if (e != cudaSuccess) return e;
    const int sms = device_info(-1).sms;
    const int per_sm = std::min(kRelMaxPerSm, std::max(1, blocks_per_sm(kern, threads, smem)));
    int64_t at_once = (int64_t)per_sm * sms;
    int cluster = 1;  // blocks a row: rows in tiles, of which there are fewer than SMs, share them out
    if (!BWD && sh.loop) {
        const int64_t tiles = (a.Lk + (int64_t)threads * sh.nv * V - 1) / ((int64_t)threads * sh.nv * V);
        while (cluster < kRelMaxCluster && cluster < tiles && p.units * cluster < sms) cluster *= 2;
        if (cluster > 1) at_once = clusters_at_once(kern, threads, cluster, smem);
        if (at_once < 1) cluster = 1, at_once = sms;
    }
    const int grid = (int)std::min<int64_t>(p.units, at_once);
    void* args[] = {&p};
    e = launch_cluster(kern, dim3(grid * cluster), dim3(threads), cluster, smem, stream, args);
    if (e != cudaSuccess) return e;
    *launches = 1;
    if (p.part) {
        e = launch_rel_table(a, grid, p.per_head, stream);
        if (e == cudaSuccess) *launches = 2;
    }
    return e;
}

}  // namespace
}  // namespace lnk
