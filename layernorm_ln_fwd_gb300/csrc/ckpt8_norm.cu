// ckpt8_norm.cu -- the LayerNorm's and RMSNorm's backward from an input kept in 8 bits.
//
// With x as the checkpoint gives it back, xhat = (x - mean) rstd (RMSNorm: mean 0) and g = gamma dy:
//   dx = rstd (g - (sum g + xhat sum g xhat) / cols)        (RMSNorm: without the first sum)
//   dgamma = sum over rows of dy xhat,  dbeta = sum over rows of dy
// ("Accelerating Transformer on GPU (II): Training with LightSeq2", section 2.1; mean and rstd are the
// forward's, of the input itself).  1 to 16 warps (a team) hold a row in registers, gamma and the column
// sums of their columns too, over all rows that they take, the next row's loads under way meanwhile.  A
// block adds its teams' column sums in order and leaves one row of partial sums for each statistic; a second,
// dependent launch adds those of a column, 32 interleaved groups and then the groups, with their rounding
// errors carried along.  No atomics: results are the same from run to run.
#include <algorithm>

#include "ckpt8.cuh"
#include "ln_finish.cuh"
#include "rel_ops.h"
#include "row_io.cuh"

namespace lnk {
namespace {

struct CnParams {
    const void* dy;
    const int8_t* q;
    const uint8_t* k;
    const void* gamma;
    const float* mean;
    const float* rstd;
    void* dx;
    float* part;   // [grid][statistics][cols]
    int rows, cols;
    Extent ed, eg;
};

template <typename T, int W, int TEAMS, int NV, bool RMS>
__global__ void __launch_bounds__(W * TEAMS * 32) ckpt_norm_kernel(const CnParams p) {
    constexpr int V = Io<T>::kVec, H = Pairs<T>::kPairs;
    constexpr int kThreads = W * TEAMS * 32;
    constexpr int NS = RMS ? 1 : 2;
    extern __shared__ float fold[];  // [NS][cols], with several teams
    __shared__ float red[2][TEAMS][2][W];
    pdl_enter();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int team = warp / W, wt = warp - team * W;
    const int cols = p.cols, blocks = ckpt_blocks(cols);
    auto column = [&](int v) { return ((v * W + wt) * 32 + lane) * V; };
    const T* DY = static_cast<const T*>(p.dy);
    uint4 gm[NV];
    f2 sg[NV][H], sb[RMS ? 1 : NV][H];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int col = column(v);
        gm[v] = col < cols ? load_columns<T>(RowIn<T>(static_cast<const T*>(p.gamma), cols, p.eg), col, cols, p.eg) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int h = 0; h < H; ++h) {
            sg[v][h] = f2_splat(0.f);
            if constexpr (!RMS) sb[v][h] = f2_splat(0.f);
        }
    }
    uint4 dn[NV];
    CkptRaw<T> qn[NV];
    float mean_n = 0.f, rstd_n = 0.f;
    auto load = [&](int64_t row) {
        rstd_n = __ldg(p.rstd + row);
        if constexpr (!RMS) mean_n = __ldg(p.mean + row);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int col = column(v);
            if (col < cols) {
                dn[v] = load_columns<T>(RowIn<T>(DY + row * cols, cols, p.ed), col, cols, p.ed);
                qn[v].load(p.q + row * blocks * kCkptBlock, p.k + row * blocks, col);
            }
        }
    };
    const int step = (int)gridDim.x * TEAMS;
    int row = (int)blockIdx.x * TEAMS + team;
    if (row < p.rows) load(row);
    const float inv = 1.0f / (float)cols;
    int parity = 0;
    for (; row < p.rows; row += step, parity ^= 1) {
        uint4 d[NV];
        CkptRaw<T> qr[NV];
        const float mean = mean_n, rstd = rstd_n;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            d[v] = dn[v];
            qr[v] = qn[v];
        }
        if (row < p.rows - step) load((int64_t)row + step);
        const f2 m2 = f2_splat(mean), r2 = f2_splat(rstd);
        f2 a = f2_splat(0.f), b = f2_splat(0.f);
        auto xhat = [&](int v, f2(&x)[H]) {
            qr[v].values(x);
#pragma unroll
            for (int h = 0; h < H; ++h) x[h] = f2_mul(RMS ? x[h] : f2_sub(x[h], m2), r2);
        };
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int col = column(v);
            if (col >= cols) continue;
            if (col + V > cols) d[v] = first_of<T>(d[v], cols - col);  // (gamma past the end times dy of 0)
            f2 x[H], dy[H], g[H];
            xhat(v, x);
            Pairs<T>::unpack(d[v], dy);
            Pairs<T>::unpack(gm[v], g);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                sg[v][h] = f2_fma(dy[h], x[h], sg[v][h]);
                if constexpr (!RMS) sb[v][h] = f2_add(sb[v][h], dy[h]);
                g[h] = f2_mul(g[h], dy[h]);
                if constexpr (!RMS) a = f2_add(a, g[h]);
                b = f2_fma(g[h], x[h], b);
            }
        }
        float sa = f2_lo(a) + f2_hi(a), sx = f2_lo(b) + f2_hi(b);
        warp_sum2(sa, sx);
        if constexpr (W > 1) {
            if (lane == 0) {
                red[parity][team][0][wt] = sa;
                red[parity][team][1][wt] = sx;
            }
            if constexpr (TEAMS == 1)
                __syncthreads();
            else
                asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(W * 32) : "memory");
            sa = sx = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                sa += red[parity][team][0][w];
                sx += red[parity][team][1][w];
            }
        }
        const f2 a2 = f2_splat(-sa * inv), b2 = f2_splat(-sx * inv);
        T* dx = static_cast<T*>(p.dx) + (int64_t)row * cols;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int col = column(v);
            if (col - lane * V >= cols) continue;  // the same in the whole warp
            uint4 u = make_uint4(0, 0, 0, 0);
            if (col < cols) {
                f2 x[H], dy[H], g[H];
                xhat(v, x);
                Pairs<T>::unpack(d[v], dy);
                Pairs<T>::unpack(gm[v], g);
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    g[h] = f2_mul(g[h], dy[h]);
                    if constexpr (!RMS) g[h] = f2_add(g[h], a2);
                    g[h] = f2_mul(r2, f2_fma(x[h], b2, g[h]));
                }
                u = Pairs<T>::pack(g);
            }
            store_columns<T>(dx, col, cols, u);
        }
    }
    // The block's column sums, its teams' in order.
    float* part = p.part + (size_t)blockIdx.x * NS * cols;
    if constexpr (TEAMS > 1) {
        for (int t = 0; t < TEAMS; ++t) {
            if (team == t) {
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const int col = column(v);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        if (col + e >= cols) continue;
                        const float s = e & 1 ? f2_hi(sg[v][e / 2]) : f2_lo(sg[v][e / 2]);
                        fold[col + e] = t ? fold[col + e] + s : s;
                        if constexpr (!RMS) {
                            const float s1 = e & 1 ? f2_hi(sb[v][e / 2]) : f2_lo(sb[v][e / 2]);
                            fold[cols + col + e] = t ? fold[cols + col + e] + s1 : s1;
                        }
                    }
                }
            }
            __syncthreads();
        }
        for (int i = tid; i < NS * cols; i += kThreads) part[i] = fold[i];
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int col = column(v);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (col + e >= cols) continue;
                part[col + e] = e & 1 ? f2_hi(sg[v][e / 2]) : f2_lo(sg[v][e / 2]);
                if constexpr (!RMS) part[cols + col + e] = e & 1 ? f2_hi(sb[v][e / 2]) : f2_lo(sb[v][e / 2]);
            }
        }
    }
}

constexpr int kCfX = 32, kCfY = 32;

template <typename T>
__global__ void __launch_bounds__(kCfX * kCfY) ckpt_norm_finish_kernel(const float* part, T* dgamma, T* dbeta,
                                                                       int blocks, int cols, int stats) {
    __shared__ float2 fold[kCfY][kCfX + 1];
    pdl_enter();
    const int n = stats * cols, c = (int)blockIdx.x * kCfX + (int)threadIdx.x;
    float s = 0.f, e = 0.f;
    if (c < n)
#pragma unroll 10
        for (int i = threadIdx.y; i < blocks; i += kCfY) comp_add(s, e, part[(size_t)i * n + c], 0.f);
    fold[threadIdx.y][threadIdx.x] = make_float2(s, e);
    __syncthreads();
    if (threadIdx.y == 0 && c < n) {
        for (int g = 1; g < kCfY; ++g) comp_add(s, e, fold[g][threadIdx.x].x, fold[g][threadIdx.x].y);
        (c < cols ? dgamma + c : dbeta + (c - cols))[0] = Io<T>::from_f(fabsf(s) < INFINITY ? s + e : s);
    }
}

struct CnShape {
    int W, teams, nv;
};
constexpr CnShape kCnShapes[] = {{1, 8, 1}, {1, 8, 2}, {1, 8, 3}, {1, 8, 4}, {2, 4, 3}, {2, 4, 4},
                                 {4, 2, 3}, {4, 2, 4}, {8, 1, 4}, {16, 1, 4}, {16, 1, 8}};
constexpr int kCnCount = sizeof(kCnShapes) / sizeof(kCnShapes[0]);

template <typename T, bool RMS>
const void* cn_kernel(int shape) {
    switch (shape) {
        case 0: return (const void*)ckpt_norm_kernel<T, 1, 8, 1, RMS>;
        case 1: return (const void*)ckpt_norm_kernel<T, 1, 8, 2, RMS>;
        case 2: return (const void*)ckpt_norm_kernel<T, 1, 8, 3, RMS>;
        case 3: return (const void*)ckpt_norm_kernel<T, 1, 8, 4, RMS>;
        case 4: return (const void*)ckpt_norm_kernel<T, 2, 4, 3, RMS>;
        case 5: return (const void*)ckpt_norm_kernel<T, 2, 4, 4, RMS>;
        case 6: return (const void*)ckpt_norm_kernel<T, 4, 2, 3, RMS>;
        case 7: return (const void*)ckpt_norm_kernel<T, 4, 2, 4, RMS>;
        case 8: return (const void*)ckpt_norm_kernel<T, 8, 1, 4, RMS>;
        case 9: return (const void*)ckpt_norm_kernel<T, 16, 1, 4, RMS>;
        default:
            if constexpr (sizeof(T) == 4) return (const void*)ckpt_norm_kernel<T, 16, 1, 8, RMS>;
            return nullptr;
    }
}

// Blocks of any shape resident on an SM at most (the registers allow fewer than 4 of 256 threads).
constexpr int kCnMaxPerSm = 4;

template <typename T, bool RMS>
cudaError_t launch_cn_t(const CkptNormArgs& a, cudaStream_t stream, int* launches) {
    constexpr int V = Io<T>::kVec;
    *launches = 0;
    const int nvec = (a.cols + V - 1) / V;
    int shape = 0;
    while (shape < kCnCount && 32 * kCnShapes[shape].W * kCnShapes[shape].nv < nvec) ++shape;
    const void* kern = shape < kCnCount ? cn_kernel<T, RMS>(shape) : nullptr;
    if (!kern) return cudaErrorInvalidValue;
    const CnShape& sh = kCnShapes[shape];
    const int threads = sh.W * sh.teams * 32;
    int stats = RMS ? 1 : 2;
    const size_t smem = sh.teams > 1 ? (size_t)stats * a.cols * sizeof(float) : 0;
    CnParams p;
    p.dy = a.dy;
    p.q = a.q;
    p.k = a.k;
    p.gamma = a.gamma;
    p.mean = a.mean;
    p.rstd = a.rstd;
    p.dx = a.dx;
    p.part = a.part;
    p.rows = a.rows;
    p.cols = a.cols;
    const char* d = static_cast<const char*>(a.dy);
    p.ed = Extent{d, d + (int64_t)a.rows * a.cols * (int64_t)sizeof(T)};
    const char* g = static_cast<const char*>(a.gamma);
    p.eg = Extent{g, g + (int64_t)a.cols * (int64_t)sizeof(T)};
    const int per_sm = std::min(kCnMaxPerSm, std::max(1, blocks_per_sm(kern, threads, smem)));
    int blocks = std::min(per_sm * device_info(-1).sms, (a.rows + sh.teams - 1) / sh.teams);
    void* args[] = {&p};
    cudaError_t e = launch_kernel(kern, dim3(blocks), dim3(threads), smem, stream, args, false);
    if (e != cudaSuccess) return e;
    const float* part = a.part;
    void *dgamma = a.dgamma, *dbeta = a.dbeta;
    int cols = a.cols;
    void* fargs[] = {&part, &dgamma, &dbeta, &blocks, &cols, &stats};
    e = launch_kernel((const void*)ckpt_norm_finish_kernel<T>, dim3((stats * cols + kCfX - 1) / kCfX),
                      dim3(kCfX, kCfY), 0, stream, fargs, false);
    if (e == cudaSuccess) *launches = 2;
    return e;
}

}  // namespace

size_t ckpt_norm_workspace_bytes(int rows, int cols, bool rms, int sms) {
    return (size_t)std::min(kCnMaxPerSm * sms, std::max(rows, 1)) * (rms ? 1 : 2) * (size_t)cols * sizeof(float);
}

cudaError_t launch_ckpt_norm_bwd(Dtype dt, const CkptNormArgs& a, cudaStream_t stream, int* launches) {
    if (dt == Dtype::F32)
        return a.mean ? launch_cn_t<float, false>(a, stream, launches) : launch_cn_t<float, true>(a, stream, launches);
    return a.mean ? launch_cn_t<__nv_bfloat16, false>(a, stream, launches)
                  : launch_cn_t<__nv_bfloat16, true>(a, stream, launches);
}

}  // namespace lnk
