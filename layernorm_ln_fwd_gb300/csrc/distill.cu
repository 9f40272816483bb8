// distill.cu -- distillation from a teacher's top logits: loss and gradient in one kernel.
//
// Per row of V student logits x with the teacher's logits t_k of the columns id_k (a negative id
// is no entry), z = scale * x, w the row's weight:
//   p_k = exp(scale t_k) / sum_k exp(scale t_k)     over the entries given,
//   log q_j = z_j - log sum_j exp z_j               over the whole row,
//   loss = w sum_k p_k (log p_k - log q_{id_k}),
//   dx_j = dloss w scale (q_j - sum_{k: id_k = j} p_k).
// Since the p_k add up to 1, with t* = max t_k, P = sum exp(scale (t_k - t*)) and the running sums
// of vocab.cuh about the reference r:
//   loss = w (scale sum_k p_k ((t_k - t*) - (x_{id_k} - r)) - log P + log Z).
#include <algorithm>
#include <math.h>

#include "ln_internal.h"
#include "vocab.cuh"

namespace lnk {
namespace {

constexpr int kDsThreads = 512;
constexpr int kDsWarps = kDsThreads / 32;
constexpr int kDsUnroll = 4;  // 128-bit loads in flight per thread in each pass

struct DsParams {
    const void* x;
    long long ld;
    const int* ids;
    const float* teacher;
    const float* weights;
    int V;
    int K;
    float scale, c;  // c = scale * log2 e
    float dloss;
    float* losses;
    void* dx;
    long long ldd;
};

struct DsShared {
    int id[LN_MAX_TOP];
    float p[LN_MAX_TOP];
    RowTotal total[kDsWarps];
    float red[2][kDsWarps];
};

__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[threadIdx.x & (kDsWarps - 1)];
#pragma unroll
    for (int o = kDsWarps / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFullMask, v, o));
    return v;
}

// Two sums over the block, the same bits in every thread.
__device__ __forceinline__ void block_sum2(float& a, float& b, float (*red)[kDsWarps]) {
    warp_sum2(a, b);
    __syncthreads();  // the last use of `red` is over
    if ((threadIdx.x & 31) == 0) {
        red[0][threadIdx.x >> 5] = a;
        red[1][threadIdx.x >> 5] = b;
    }
    __syncthreads();
    sum_warp_values2(red[0], red[1], kDsWarps, a, b);
}

// One block a row.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(kDsThreads, 2) distill_kernel(const DsParams p) {
    using IO = Io<T>;
    using PR = Pairs<T>;
    constexpr int kVec = IO::kVec;
    constexpr int H = PR::kPairs;
    __shared__ DsShared sh;
    const int tid = (int)threadIdx.x;
    pdl_enter();
    const size_t row = blockIdx.x;
    const T* xr = static_cast<const T*>(p.x) + row * (size_t)p.ld;
    T* dr = p.dx ? static_cast<T*>(p.dx) + row * (size_t)p.ldd : nullptr;
    const RowCut<T> cut(xr, p.V);
    const uint4* xv = reinterpret_cast<const uint4*>(xr + cut.head);
    const int nvec = cut.nvec;
    // The teacher's weights.  Entry k is thread k's.
    int id = -1;
    float t = -INFINITY;
    if (tid < p.K) {
        id = p.ids[row * (size_t)p.K + tid];
        if (id >= 0) t = p.teacher[row * (size_t)p.K + tid];
        sh.id[tid] = id;
    }
    const float w = p.weights ? p.weights[row] : 1.f;
    const bool bad = __syncthreads_or(id >= p.V);
    const bool odd = __syncthreads_or(t != t);
    const float tmax = block_max(t, sh.red[0]);
    if ((tmax == -INFINITY && !odd && !bad) || w == 0.f) {
        // Nothing to learn from: no entry, or a row that does not count.  The row is not read.
        if (tid == 0 && p.losses) p.losses[row] = 0.f;
        if (dr) {
            if constexpr (WIDE) {
                for (int v = tid; v < nvec; v += kDsThreads)
                    st_stream(dr + cut.col(v), make_uint4(0, 0, 0, 0));
                if (tid < cut.nloose()) dr[cut.loose(tid)] = IO::from_f(0.f);
            } else {
                for (int j = tid; j < p.V; j += kDsThreads) dr[j] = IO::from_f(0.f);
            }
        }
        return;
    }
    const bool mine = id >= 0 && id < p.V;
    const float xk = mine ? IO::to_f(xr[id]) : 0.f;
    // Pass 1: the row's sums.
    RowSums<false> s;
    s.clear();
    const f2 c2 = f2_splat(p.c);
    for (int v0 = tid; v0 < nvec; v0 += kBatch * kDsThreads) {
        uint4 u[kBatch];
        load_batch<T>(u, xv, v0, kDsThreads, nvec);
        if (s.see_batch<T>(u, p.c) > -INFINITY)
            s.add_batch<T>(u, c2, [&](int k) { return u[k]; });
    }
    if (tid < cut.nloose()) s.add_one(IO::to_f(xr[cut.loose(tid)]), p.c);
    const RowTotal a = block_total({s.ref, f2_lo(s.z2) + f2_hi(s.z2), 0.f}, p.c, sh.total);
    const float r = a.ref == -INFINITY ? 0.f : a.ref;
    // The teacher's sum, then what its weights make of its logits and the student's.
    const float e = id >= 0 ? ex2_fast((t - tmax) * p.c) : 0.f;
    float esum = e, none = 0.f;
    block_sum2(esum, none, sh.red);
    const float pk = e / esum;
    // An entry of weight 0 adds nothing, whatever the student has there.
    float gap = pk != 0.f ? pk * ((t - tmax) - (xk - r)) : 0.f;
    none = 0.f;
    block_sum2(gap, none, sh.red);
    const float nan = __int_as_float(0x7fc00000);
    if (tid == 0 && p.losses)
        p.losses[row] = bad ? nan : w * (fmaf(gap, p.scale, -logf(esum)) + logf(a.z));
    if (!dr) return;
    if (tid < p.K) sh.p[tid] = pk;
    // Pass 2: the gradient, the columns of the teacher's entries last.
    const float co = bad ? nan : p.dloss * w * p.scale;
    const float cz = co / a.z;
    const f2 r2 = f2_splat(-r), cz2 = f2_splat(cz);
    for (int v0 = tid; v0 < nvec; v0 += kDsUnroll * kDsThreads) {
        uint4 u[kDsUnroll];
#pragma unroll
        for (int k = 0; k < kDsUnroll; ++k) {
            const int v = v0 + k * kDsThreads;
            if (v < nvec) u[k] = __ldcs(xv + v);
        }
#pragma unroll
        for (int k = 0; k < kDsUnroll; ++k) {
            const int v = v0 + k * kDsThreads;
            if (v >= nvec) break;
            f2 x2[H], o[H];
            PR::unpack(u[k], x2);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const f2 z = f2_mul(f2_add(x2[h], r2), c2);
                o[h] = f2_mul(f2_make(ex2_fast(f2_lo(z)), ex2_fast(f2_hi(z))), cz2);
            }
            if constexpr (WIDE) {
                st_stream(dr + cut.col(v), PR::pack(o));
            } else {
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    dr[cut.col(v) + 2 * h] = IO::from_f(f2_lo(o[h]));
                    dr[cut.col(v) + 2 * h + 1] = IO::from_f(f2_hi(o[h]));
                }
            }
        }
    }
    if (tid < cut.nloose()) {
        const int col = cut.loose(tid);
        dr[col] = IO::from_f(ex2_fast((IO::to_f(xr[col]) - r) * p.c) * cz);
    }
    __syncthreads();  // the whole row is written; sh.p
    if (mine) {
        // One writer a column: the first of the entries that name it, with all their weights.
        float sum = 0.f;
        bool first = true;
        for (int k = 0; k < p.K; ++k) {
            if (sh.id[k] != id) continue;
            if (k < tid) first = false;
            sum += sh.p[k];
        }
        if (first) dr[id] = IO::from_f(fmaf(ex2_fast((xk - r) * p.c), cz, -co * sum));
    }
}

template <typename T>
cudaError_t launch_distill_t(const DistillArgs& a, cudaStream_t stream) {
    DsParams p;
    p.x = a.logits;
    p.ld = a.ld;
    p.ids = a.ids;
    p.teacher = a.teacher;
    p.weights = a.weights;
    p.V = a.V;
    p.K = a.K;
    p.scale = a.scale;
    p.c = a.scale * kLog2e;
    p.dloss = a.dloss;
    p.losses = a.losses;
    p.dx = a.dlogits;
    p.ldd = a.ldd;
    const bool wide = !a.dlogits || rows_congruent(a.logits, a.ld, a.dlogits, a.ldd, sizeof(T), a.rows);
    const void* kern = wide ? (const void*)distill_kernel<T, true> : (const void*)distill_kernel<T, false>;
    void* args[] = {&p};
    return launch_kernel(kern, dim3((unsigned)a.rows), dim3(kDsThreads), 0, stream, args, false);
}

}  // namespace

cudaError_t launch_distill(Dtype dt, const DistillArgs& a, cudaStream_t stream, int* launches) {
    cudaError_t e = dt == Dtype::F32 ? launch_distill_t<float>(a, stream)
                                     : launch_distill_t<__nv_bfloat16>(a, stream);
    *launches = e == cudaSuccess;
    return e;
}

}  // namespace lnk
