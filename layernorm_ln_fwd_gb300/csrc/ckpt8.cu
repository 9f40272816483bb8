// ckpt8.cu -- 8-bit checkpoints of activations: rows to integers and steps (ckpt8.cuh has the format), and back.
//
// A warp takes 32 vectors of 16 bytes of a row at a time, several of them in flight; aligned rows of whole blocks that
// follow one another are taken as one long row, without arithmetic on rows (bf16 8192 x 4096 there and back 47 -> 30 us,
// the measured copy rate).  Narrow rows are taken by 8 or 16 lanes each (bf16 65536 x 40 there and back 14 us; by a
// warp, four fifths of it idle, 30).  Bound by memory: each value is read once and written once; odd rows (65536 x 1001 104
// us, 0.56 of the copy rate) by the words at their ends and by the stores put together from two lanes.
#include <algorithm>

#include "ckpt8.cuh"
#include "rel_ops.h"
#include "row_io.cuh"

namespace lnk {
namespace {

constexpr int kCkThreads = 256;
constexpr int kCkFlight = 4;  // a warp's pieces of rows in flight

struct CkParams {
    const void* x;   // store
    void* out;       // load
    int64_t ld, rows, cols, segs, total;
    int64_t ldq, ldk;
    int8_t* q;
    uint8_t* k;
    Extent ex;
};

// Aligned rows of whole blocks that follow one another, as one: piece `at` of 32 vectors, of `cols` in all.
template <typename T, bool STORE>
__global__ void __launch_bounds__(kCkThreads) ckpt8_flat_kernel(const CkParams p) {
    constexpr int V = Io<T>::kVec, S = 32 * V, F = STORE ? kCkFlight : 2 * kCkFlight;
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kCkThreads / 32);
    const int64_t w0 = (int64_t)blockIdx.x * (kCkThreads / 32) + (threadIdx.x >> 5);
    for (int64_t base = w0; base < p.total; base += warps * F) {
        uint4 u[STORE ? F : 1];
        CkptRaw<T> raw[STORE ? 1 : F];
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const int64_t col = (base + f * warps) * S + lane * V;
            if (col >= p.cols) continue;
            if constexpr (STORE)
                u[f] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + col));
            else
                raw[f].load(p.q + (col - lane * V), p.k + (col - lane * V) / kCkptBlock, lane * V);
        }
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const int64_t from = (base + f * warps) * S;
            if (from >= p.cols) break;  // the same in the whole warp
            const bool mine = from + lane * V < p.cols;
            if constexpr (STORE) {
                if (!mine) u[f] = make_uint4(0, 0, 0, 0);
                ckpt_keep<T>(u[f], lane * V, (int)min((int64_t)S, p.cols - from), p.q + from, p.k + from / kCkptBlock);
            } else if (mine) {
                f2 v[Pairs<T>::kPairs];
                raw[f].values(v);
                st_stream(static_cast<T*>(p.out) + from + lane * V, Pairs<T>::pack(v));
            }
        }
    }
}

// Rows of any kind: L lanes (fewer than 32 for narrow rows) take kCkFlight pieces of L vectors of a row that follow
// one another.
template <typename T, bool STORE, int L>
__global__ void __launch_bounds__(kCkThreads) ckpt8_kernel(const CkParams p) {
    constexpr int V = Io<T>::kVec, S = L * V, G = kCkThreads / L;
    pdl_enter();
    const int lane = threadIdx.x & (L - 1);
    const int64_t groups = (int64_t)gridDim.x * G;
    for (int64_t at0 = (int64_t)blockIdx.x * G + (threadIdx.x & ~31u) / L; at0 < p.total; at0 += groups) {
        // (A warp's groups together: one past the last takes the last again, and stores nothing.)
        const int64_t mine = at0 + (threadIdx.x & 31) / L, at = min(mine, p.total - 1);
        const bool ok = L == 32 || mine < p.total;
        const int64_t row = at / p.segs;
        const int cols = (int)p.cols, from = (int)(at - row * p.segs) * kCkFlight * S + lane * V;
        int8_t* q = p.q + row * p.ldq;
        uint8_t* k = p.k + row * p.ldk;
        if constexpr (STORE) {
            const RowIn<T> in(static_cast<const T*>(p.x) + row * p.ld, cols, p.ex);
            uint4 u[kCkFlight];
#pragma unroll
            for (int f = 0; f < kCkFlight; ++f) {
                const int col = from + f * S;
                u[f] = col < cols ? load_columns<T>(in, col, cols, p.ex) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int f = 0; f < kCkFlight; ++f) {
                const int col = from + f * S;
                if (L == 32 && col - lane * V >= cols) break;  // the same in the whole warp
                if (col < cols && col + V > cols) u[f] = first_of<T>(u[f], cols - col);
                ckpt_keep<T>(u[f], col, ok ? ckpt_blocks(cols) * kCkptBlock : 0, q, k);
            }
        } else {
            CkptRaw<T> raw[kCkFlight];
#pragma unroll
            for (int f = 0; f < kCkFlight; ++f) {
                raw[f].clear();
                if (from + f * S < cols) raw[f].load(q, k, from + f * S);
            }
            RowOut<T, L> out;
#pragma unroll
            for (int f = 0; f < kCkFlight; ++f) {
                const int col = from + f * S;
                if (L == 32 && col - lane * V >= cols) break;  // the same in the whole warp
                f2 v[Pairs<T>::kPairs];
                raw[f].values(v);
                out.put(static_cast<T*>(p.out) + row * p.ld, col, ok ? cols : 0, Pairs<T>::pack(v), f == 0, f == kCkFlight - 1);
            }
        }
    }
}

template <typename T, bool STORE>
cudaError_t launch_t(CkParams p, cudaStream_t stream) {
    constexpr int S = 32 * Io<T>::kVec;
    p.ldk = ckpt_blocks((int)p.cols);
    p.ldq = p.ldk * kCkptBlock;
    const char* base = static_cast<const char*>(p.x);
    p.ex = Extent{base, base ? base + ((p.rows - 1) * p.ld + p.cols) * (int64_t)sizeof(T) : base};
    const void* t = STORE ? p.x : p.out;
    const bool flat = p.cols == p.ldq && p.ld == p.cols && (reinterpret_cast<uintptr_t>(t) & 15u) == 0;
    if (flat) {
        p.cols *= p.rows;
        p.rows = 1;
    }
    const int64_t vectors = (p.cols + S / 32 - 1) / (S / 32);
    const int lanes = flat || vectors > 16 * kCkFlight ? 32 : vectors > 8 * kCkFlight ? 16 : 8;
    const int64_t per = flat ? S : (int64_t)kCkFlight * (S / 32) * lanes;
    p.segs = (p.cols + per - 1) / per;
    p.total = p.segs * p.rows;
    const void* kern = flat          ? (const void*)ckpt8_flat_kernel<T, STORE>
                       : lanes == 32 ? (const void*)ckpt8_kernel<T, STORE, 32>
                       : lanes == 16 ? (const void*)ckpt8_kernel<T, STORE, 16>
                                     : (const void*)ckpt8_kernel<T, STORE, 8>;
    const int64_t slots = (int64_t)std::max(1, blocks_per_sm(kern, kCkThreads, 0)) * device_info(-1).sms;
    const int64_t each = kCkThreads / lanes, need = (p.total + each - 1) / each;
    void* args[] = {&p};
    return launch_kernel(kern, dim3((unsigned)std::min(slots, need)), dim3(kCkThreads), 0, stream, args, false);
}

}  // namespace

cudaError_t launch_ckpt8_store(Dtype dt, const void* x, int64_t ld, int64_t rows, int cols, int8_t* q,
                               uint8_t* k, cudaStream_t stream) {
    CkParams p = {};
    p.x = x;
    p.ld = ld;
    p.rows = rows;
    p.cols = cols;
    p.q = q;
    p.k = k;
    return dt == Dtype::F32 ? launch_t<float, true>(p, stream) : launch_t<__nv_bfloat16, true>(p, stream);
}

cudaError_t launch_ckpt8_load(Dtype dt, const int8_t* q, const uint8_t* k, int64_t rows, int cols, void* x,
                              int64_t ld, cudaStream_t stream) {
    CkParams p = {};
    p.out = x;
    p.ld = ld;
    p.rows = rows;
    p.cols = cols;
    p.q = const_cast<int8_t*>(q);
    p.k = const_cast<uint8_t*>(k);
    return dt == Dtype::F32 ? launch_t<float, false>(p, stream) : launch_t<__nv_bfloat16, false>(p, stream);
}

}  // namespace lnk
