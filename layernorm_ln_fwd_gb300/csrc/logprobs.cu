// logprobs.cu -- log probabilities of given tokens over rows of logits, with the entropy, the
// token's rank and the top alternatives, and the gradient of the log probability and the entropy.
//
// Per row of V logits x with token t, z = scale * x:
//   L = log sum_j exp z_j,  q_j = exp(z_j - L),  logp = z_t - L,  H = -sum_j q_j log q_j,
//   dx_j = scale (dlogp (1[j = t] - q_j) - dH q_j (log q_j + H)).
// With u = (x - r) scale log2 e about a reference r (vocab.cuh), Z = sum 2^u and W = sum 2^u u:
//   L = scale r + log Z,   log q_j = (x_j - r) scale - log Z,   H = log Z - ln 2 W / Z.
#include <algorithm>
#include <math.h>

#include "ln_internal.h"
#include "top_select.cuh"
#include "vocab.cuh"

namespace lnk {
namespace {

constexpr int kLpMaxThreads = 512;
constexpr int kLpUnroll = 4;        // 128-bit loads in flight per thread
constexpr int kLpSegments = 2048;   // segments of a row at most (and one thread's share more)
constexpr int kLpCand = 4096;       // candidates held at once
constexpr int kLpFlagged = 2 * LN_MAX_TOP;
constexpr int kLpLoose = 16;        // at least 2 * (kVec - 1) loose elements of a row

struct LpParams {
    const void* x;
    long long ld;
    const int* tokens;
    int V;
    int top;
    int seglen;   // vectors of a thread that share a segment
    int nseg;     // segments of vectors: a multiple of the block's threads
    float scale, c;  // c = scale * log2 e
    float* logp;
    float* entropy;
    float* lse;
    int* ranks;
    int* top_ids;
    float* top_logp;
};

struct TopShared {
    SelectShared sel;
    entry_t cand[kLpCand];
    entry_t keep[LN_MAX_TOP];
    int flagged[kLpFlagged];
    int nflag, ncand;
    // entry_t segs[nseg + kLpLoose] follows
};

// The top entries of a row whose segments' largest entries are in `segs`.
//
// While the row streams by, nothing is done for the top but to keep the largest value of each
// segment (a few vectors of one thread) and the vector that first held it.  The k-th largest of
// these entries is a lower bound of the row's k-th largest element: k different vectors hold an
// element that is as large.  So only segments whose largest entry reaches the bound can hold a
// top element -- k of them, or a few more for a bound found with some slack -- and those alone are
// read again (k * seglen vectors of a row that has just been read, from L2), their elements that
// reach the bound becoming the candidates.  An element equal in value to the bound counts only
// in a vector no later than the bound's, so that rows of many equal values (constant rows, rows
// masked by the type's lowest value) have few candidates too.
//
// Returns the number of entries left in *list (shared memory, in no order), all of the top among
// them.
template <typename T>
__device__ __forceinline__ int collect_top(const LpParams& p, const uint4* xv, int nvec, int head,
                                           TopShared* sh, const entry_t* segs, const entry_t** list) {
    using IO = Io<T>;
    constexpr int kVec = IO::kVec;
    const int tid = (int)threadIdx.x, nt = (int)blockDim.x, k = p.top;
    if (tid == 0) sh->nflag = sh->ncand = 0;
    __syncthreads();
    const int nall = p.nseg + kLpLoose;
    const entry_t bound = select_threshold(segs, nall, k, k / 4 + 16, &sh->sel);
    const float least = bound == 1 ? -3.402823466e38f : entry_value(bound);
    for (int i = tid; i < nall; i += nt) {
        const entry_t e = segs[i];
        if (e < bound) continue;
        if (i < p.nseg)
            sh->flagged[atomicAdd(&sh->nflag, 1)] = i;  // at most k + k / 4 + 16 < kLpFlagged
        else
            sh->cand[atomicAdd(&sh->ncand, 1)] = e;  // a loose element is a segment of its own
    }
    __syncthreads();
    const int items = sh->nflag * p.seglen;
    auto vector_of = [&](int w) {
        const int seg = sh->flagged[w / p.seglen];
        return seg % nt + nt * (seg / nt * p.seglen + w % p.seglen);
    };
    for (int w = tid; w < items; w += nt) {
        const int v = vector_of(w);
        if (v >= nvec) continue;
        const uint4 u = __ldcg(xv + v);
        if (!(vector_max<T>(u) >= least)) continue;
        float f[kVec];
        IO::unpack(u, f);
        const int col = head + v * kVec;
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (f[j] >= least && make_entry(f[j], col) >= bound) {
                const int at = atomicAdd(&sh->ncand, 1);
                if (at < kLpCand) sh->cand[at] = make_entry(f[j], col + j);
            }
    }
    __syncthreads();
    int n = sh->ncand;
    auto keep_top = [&](int have) {  // the top k of cand[0 .. have) into keep, in no order
        const entry_t t = select_threshold(sh->cand, have, k, 0, &sh->sel);
        if (tid == 0) sh->ncand = 0;
        __syncthreads();
        for (int i = tid; i < have; i += nt)
            if (sh->cand[i] >= t) sh->keep[atomicAdd(&sh->ncand, 1)] = sh->cand[i];
        __syncthreads();
        return t;
    };
    if (n > kLpCand) {
        // More candidates than there is room for: few segments hold very many large values.  Go
        // through them again one element a thread at a time, cutting down to the top k whenever
        // the next step might not fit.
        entry_t floor_e = 0;
        __syncthreads();
        if (tid == 0) sh->ncand = 0;
        __syncthreads();
        for (int w0 = 0; w0 < items + kLpLoose; w0 += nt) {
            const int w = w0 + tid;
            uint4 u = make_uint4(0, 0, 0, 0);
            int col = -1;
            if (w < items) {
                const int v = vector_of(w);
                if (v < nvec) {
                    u = __ldcg(xv + v);
                    col = head + v * kVec;
                }
            }
            float f[kVec];
            IO::unpack(u, f);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                entry_t e = 0;
                if (col >= 0) {
                    if (f[j] >= least && make_entry(f[j], col) >= bound) e = make_entry(f[j], col + j);
                } else if (j == 0 && w >= items && w < items + kLpLoose) {
                    e = segs[p.nseg + (w - items)];
                    if (e < bound) e = 0;
                }
                if (e > floor_e) sh->cand[atomicAdd(&sh->ncand, 1)] = e;
                __syncthreads();
                const int have = sh->ncand;
                __syncthreads();
                if (have > kLpCand - nt) {
                    floor_e = keep_top(have) - 1;  // entries below the k-th are out for good
                    const int kept = sh->ncand;
                    for (int i = tid; i < kept; i += nt) sh->cand[i] = sh->keep[i];
                    __syncthreads();
                }
            }
        }
        n = sh->ncand;
    }
    if (n <= 2 * LN_MAX_TOP) {  // few enough to be put in order by counting
        *list = sh->cand;
        return n;
    }
    keep_top(n);
    *list = sh->keep;
    return sh->ncand;
}

// One block a row.  The row is read once, kLpUnroll vectors of a thread in flight at a time.
template <typename T, bool ENT, bool TOP>
__global__ void __launch_bounds__(kLpMaxThreads, 2) logprobs_kernel(const LpParams p) {
    using IO = Io<T>;
    using PR = Pairs<T>;
    constexpr int kVec = IO::kVec;
    constexpr int H = PR::kPairs;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __shared__ RowTotal sh_total[kLpMaxThreads / 32];
    __shared__ int sh_above;
    TopShared* sh = reinterpret_cast<TopShared*>(smem_raw);
    entry_t* segs = reinterpret_cast<entry_t*>(smem_raw + sizeof(TopShared));
    const int tid = (int)threadIdx.x, nt = (int)blockDim.x;
    pdl_enter();
    const size_t row = blockIdx.x;
    const T* xr = static_cast<const T*>(p.x) + row * (size_t)p.ld;
    const RowCut<T> cut(xr, p.V);
    const uint4* xv = reinterpret_cast<const uint4*>(xr + cut.head);
    const int nvec = cut.nvec;
    const int t = p.tokens ? p.tokens[row] : -1;
    const bool has = t >= 0 && t < p.V;
    const float xt = has ? IO::to_f(xr[t]) : __int_as_float(0x7fc00000);
    const float over = p.ranks ? xt : __int_as_float(0x7fc00000);  // values above it are counted
    if (tid == 0) sh_above = 0;
    RowSums<ENT> s;
    s.clear();
    const f2 c2 = f2_splat(p.c);
    int above = 0;
    float best = -INFINITY;
    int bestv = 0, left = p.seglen, seg = tid;
    for (int v0 = tid; v0 < nvec; v0 += kLpUnroll * nt) {
        uint4 u[kLpUnroll];
#pragma unroll
        for (int k = 0; k < kLpUnroll; ++k) {
            const int v = v0 + k * nt;
            if (v < nvec) u[k] = __ldcg(xv + v);
        }
#pragma unroll
        for (int k = 0; k < kLpUnroll; ++k) {
            const int v = v0 + k * nt;
            if (v >= nvec) break;
            const float m = vector_max<T>(u[k]);
            s.see(m, p.c);
            f2 x2[H];
            PR::unpack(u[k], x2);
            s.add(x2, c2);
            if (m > over) {
#pragma unroll
                for (int h = 0; h < H; ++h) above += (f2_lo(x2[h]) > over) + (f2_hi(x2[h]) > over);
            }
            if constexpr (TOP) {
                if (m > best) {
                    best = m;
                    bestv = v;
                }
                if (--left == 0) {
                    segs[seg] = best > -INFINITY ? make_entry(best, cut.col(bestv)) : 0;
                    seg += nt;
                    best = -INFINITY;
                    left = p.seglen;
                }
            }
        }
    }
    if constexpr (TOP) {
        for (; seg < p.nseg; seg += nt) {  // the last, unfilled segment, and those of no vector
            segs[seg] = best > -INFINITY ? make_entry(best, cut.col(bestv)) : 0;
            best = -INFINITY;
        }
        if (tid < kLpLoose) segs[p.nseg + tid] = 0;
    }
    if (tid < cut.nloose()) {
        const int col = cut.loose(tid);
        const float x = IO::to_f(xr[col]);
        s.add_one(x, p.c);
        above += x > over;
        if constexpr (TOP)
            if (x > -INFINITY) segs[p.nseg + tid] = make_entry(x, col);
    }
    RowTotal mine{s.ref, f2_lo(s.z2) + f2_hi(s.z2), ENT ? f2_lo(s.w2) + f2_hi(s.w2) : 0.f};
    __syncthreads();  // sh_above, segs
    above = __reduce_add_sync(kFullMask, above);
    if ((tid & 31) == 0 && above) atomicAdd(&sh_above, above);
    const RowTotal a = block_total(mine, p.c, sh_total);
    __syncthreads();
    const float r = a.ref == -INFINITY ? 0.f : a.ref;
    const float logz = logf(a.z);
    if (tid == 0) {
        if (p.lse) p.lse[row] = fmaf(r, p.scale, logz);
        if (ENT) p.entropy[row] = logz - kLn2 * a.w / a.z;
        if (p.tokens) {
            // No token (t < 0): 0, of rank 0.  A token outside the row: NaN, of rank 0.
            if (p.logp) p.logp[row] = t < 0 ? 0.f : fmaf(xt - r, p.scale, -logz);
            if (p.ranks) p.ranks[row] = has ? sh_above + 1 : 0;
        }
    }
    if constexpr (TOP) {
        const entry_t* list;
        const int n = collect_top<T>(p, xv, nvec, cut.head, sh, segs, &list);
        int* ids = p.top_ids + row * (size_t)p.top;
        float* lp = p.top_logp + row * (size_t)p.top;
        for (int i = tid; i < n; i += nt) {
            const entry_t e = list[i];
            const int at = place_of(e, list, n);
            if (at < p.top) {
                ids[at] = entry_col(e);
                lp[at] = fmaf(entry_value(e) - r, p.scale, -logz);
            }
        }
        for (int i = n + tid; i < p.top; i += nt) {  // fewer logits above -inf than places
            ids[i] = -1;
            lp[i] = -INFINITY;
        }
    }
}

template <typename T>
cudaError_t launch_logprobs_t(const LogprobsArgs& a, cudaStream_t stream) {
    constexpr int kVec = Io<T>::kVec;
    LpParams p;
    p.x = a.logits;
    p.ld = a.ld;
    p.tokens = a.tokens;
    p.V = a.V;
    p.top = a.top;
    p.scale = a.scale;
    p.c = a.scale * kLog2e;
    p.logp = a.logp;
    p.entropy = a.entropy;
    p.lse = a.lse;
    p.ranks = a.ranks;
    p.top_ids = a.top_ids;
    p.top_logp = a.top_logp;
    const int nvec = a.V / kVec;
    const int nt = nvec >= 2048 ? 512 : nvec >= 512 ? 256 : 128;
    const int per = std::max(1, (nvec + nt - 1) / nt);  // vectors of a thread
    p.seglen = std::max(1, (per * nt + kLpSegments - 1) / kLpSegments);
    p.nseg = (per + p.seglen - 1) / p.seglen * nt;
    const bool top = a.top > 0, ent = a.entropy != nullptr;
    const size_t smem = top ? sizeof(TopShared) + ((size_t)p.nseg + kLpLoose) * sizeof(entry_t) : 0;
    const void* kern = top ? (ent ? (const void*)logprobs_kernel<T, true, true>
                                  : (const void*)logprobs_kernel<T, false, true>)
                           : (ent ? (const void*)logprobs_kernel<T, true, false>
                                  : (const void*)logprobs_kernel<T, false, false>);
    if (top) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    void* args[] = {&p};
    return launch_kernel(kern, dim3((unsigned)a.rows), dim3(nt), smem, stream, args, false);
}

// ---------------------------------------------------------------------------------------
// The gradient.  The forward left L and H, so every element stands for itself: one warp takes a
// piece of a row (kLbUnroll vectors a lane), reads it, and writes the gradient of the same
// elements, which may be the logits' own place.
// ---------------------------------------------------------------------------------------
constexpr int kLbThreads = 256;
constexpr int kLbUnroll = 4;

struct LbParams {
    const void* x;
    long long ld;
    const int* tokens;
    const float* lse;
    const float* entropy;
    const float* dlogp;
    const float* dent;
    long long pieces;  // rows * per_row
    int per_row;
    int V;
    float scale;
    void* dx;
    long long ldd;
};

// WIDE: logits and gradient lie at the same place of a 16-byte vector in every row.
template <typename T, bool ENT, bool WIDE>
__global__ void __launch_bounds__(kLbThreads) logprobs_bwd_kernel(const LbParams p) {
    using IO = Io<T>;
    constexpr int kVec = IO::kVec;
    pdl_enter();
    const int lane = (int)threadIdx.x & 31;
    const long long piece = (long long)blockIdx.x * (kLbThreads / 32) + (threadIdx.x >> 5);
    if (piece >= p.pieces) return;
    const size_t row = (size_t)(piece / p.per_row);
    const int part = (int)(piece % p.per_row);
    const T* xr = static_cast<const T*>(p.x) + row * (size_t)p.ld;
    T* dr = static_cast<T*>(p.dx) + row * (size_t)p.ldd;
    const RowCut<T> cut(xr, p.V);
    const int t = p.tokens ? p.tokens[row] : -1;
    const bool bad = p.dlogp && t >= p.V;
    float g = p.dlogp && t >= 0 ? p.dlogp[row] : 0.f;
    const float de = ENT ? p.dent[row] : 0.f;
    const bool none = g == 0.f && de == 0.f;  // nothing flows back: 0, whatever the row holds
    if (bad) g = __int_as_float(0x7fc00000);
    const float lse = p.lse[row], hh = ENT ? p.entropy[row] : 0.f;
    const float sg = p.scale * g, sde = p.scale * de;
    auto grad = [&](float x, int col) {
        const float logq = fmaf(x, p.scale, -lse);
        const float q = ex2_fast(logq * kLog2e);
        float o = -sg * q;
        if constexpr (ENT) o = fmaf(-sde * q, fmaxf(logq, -1e30f) + hh, o);
        return col == t ? o + sg : o;
    };
    const int lo = (int)((long long)cut.nvec * part / p.per_row);
    const int hi = (int)((long long)cut.nvec * (part + 1) / p.per_row);
    const uint4* xv = reinterpret_cast<const uint4*>(xr + cut.head);
    for (int v0 = lo + lane; v0 < hi; v0 += 32 * kLbUnroll) {
        uint4 u[kLbUnroll];
#pragma unroll
        for (int k = 0; k < kLbUnroll; ++k) {
            const int v = v0 + 32 * k;
            u[k] = v < hi && !none ? __ldcs(xv + v) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < kLbUnroll; ++k) {
            const int v = v0 + 32 * k;
            if (v >= hi) break;
            const int col = cut.col(v);
            float f[kVec];
            IO::unpack(u[k], f);
#pragma unroll
            for (int j = 0; j < kVec; ++j) f[j] = none ? 0.f : grad(f[j], col + j);
            if constexpr (WIDE) {
                st_stream(dr + col, IO::pack(f));
            } else {
#pragma unroll
                for (int j = 0; j < kVec; ++j) dr[col + j] = IO::from_f(f[j]);
            }
        }
    }
    if (part == 0 && lane < cut.nloose()) {
        const int col = cut.loose(lane);
        dr[col] = IO::from_f(none ? 0.f : grad(IO::to_f(xr[col]), col));
    }
}

template <typename T>
cudaError_t launch_logprobs_bwd_t(const LogprobsBwdArgs& a, cudaStream_t stream) {
    constexpr int kVec = Io<T>::kVec;
    LbParams p;
    p.x = a.logits;
    p.ld = a.ld;
    p.tokens = a.tokens;
    p.lse = a.lse;
    p.entropy = a.entropy;
    p.dlogp = a.dlogp;
    p.dent = a.dentropy;
    p.V = a.V;
    p.scale = a.scale;
    p.dx = a.dlogits;
    p.ldd = a.ldd;
    const int nvec = a.V / kVec;
    p.per_row = std::max(1, (nvec + 32 * kLbUnroll - 1) / (32 * kLbUnroll));
    p.pieces = (long long)a.rows * p.per_row;
    const bool wide = rows_congruent(a.logits, a.ld, a.dlogits, a.ldd, sizeof(T), a.rows);
    const bool ent = a.dentropy != nullptr;
    const void* kern = ent ? (wide ? (const void*)logprobs_bwd_kernel<T, true, true>
                                   : (const void*)logprobs_bwd_kernel<T, true, false>)
                           : (wide ? (const void*)logprobs_bwd_kernel<T, false, true>
                                   : (const void*)logprobs_bwd_kernel<T, false, false>);
    const long long blocks = (p.pieces + kLbThreads / 32 - 1) / (kLbThreads / 32);
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    void* args[] = {&p};
    return launch_kernel(kern, dim3((unsigned)blocks), dim3(kLbThreads), 0, stream, args, false);
}

}  // namespace

bool rows_congruent(const void* a, int64_t lda, const void* b, int64_t ldb, size_t esize, int rows) {
    const uint64_t base = reinterpret_cast<uintptr_t>(a) - reinterpret_cast<uintptr_t>(b);
    if (base & 15u) return false;
    return rows < 2 || (((uint64_t)lda - (uint64_t)ldb) * esize & 15u) == 0;
}

cudaError_t launch_logprobs(Dtype dt, const LogprobsArgs& a, cudaStream_t stream, int* launches) {
    cudaError_t e = dt == Dtype::F32 ? launch_logprobs_t<float>(a, stream)
                                     : launch_logprobs_t<__nv_bfloat16>(a, stream);
    *launches = e == cudaSuccess;
    return e;
}

cudaError_t launch_logprobs_bwd(Dtype dt, const LogprobsBwdArgs& a, cudaStream_t stream,
                                int* launches) {
    cudaError_t e = dt == Dtype::F32 ? launch_logprobs_bwd_t<float>(a, stream)
                                     : launch_logprobs_bwd_t<__nv_bfloat16>(a, stream);
    *launches = e == cudaSuccess;
    return e;
}

}  // namespace lnk
