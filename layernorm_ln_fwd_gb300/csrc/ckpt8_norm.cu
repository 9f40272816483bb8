// ckpt8_norm.cu -- the LayerNorm's and RMSNorm's backward from an input kept in 8 bits.
//
// With x as the checkpoint gives it back, xhat = (x - mean) rstd (RMSNorm: mean 0) and g = gamma dy:
//   dx = rstd (g - (sum g + xhat sum g xhat) / cols)        (RMSNorm: without the first sum)
//   dgamma = sum over rows of dy xhat,  dbeta = sum over rows of dy
// ("Accelerating Transformer on GPU (II): Training with LightSeq2", section 2.1; mean and rstd are the
// forward's, of the input itself).  A row is held by 1 to 16 warps (a team), at 4 to 32 columns a lane,
// and each lane keeps the column sums of its columns over all rows that its team takes.  dy and the integers of
// the next 1 to 3 rows are on their way meanwhile, by asynchronous copies of 16 and 8 (4) bytes into
// shared memory that each lane makes and reads for itself, without barriers.  A block adds its teams' column sums in
// order and leaves one row of partial sums for each statistic; a second, dependent launch adds those of a column,
// 32 interleaved groups and then the groups, with their rounding errors carried along.  No atomics: results are the
// same from run to run.
//
// LayerNorm, bf16 65536 x 768: 53 us, 0.70 of the measured copy rate; RMSNorm 4096 x 8192 38.7 us, 0.64, fp32 4096 x 4096 32
// us, 0.69.  Small calls (8192 x 768: 12.5 us for 4.7 of traffic) are bound by what comes once: the first rows' way, a
// block's column sums, the second launch.  LayerNorm beyond 24 columns a lane (bf16 4096 x 8192: 52 us, 0.48) by the second
// conversion of its integers, for which two column sums leave no registers.
#include <algorithm>
#include <utility>

#include "ckpt8.cuh"
#include "ln_finish.cuh"
#include "rel_ops.h"
#include "row_io.cuh"

namespace lnk {
namespace {

// Rows of a team in shared memory or on their way there: 3, in fp32 2, where they fit beside gamma.  More do no
// good: LayerNorm, bf16 65536 x 768, with 2, 3, 4: 54.5, 53.1, 53.8 us; 65536 x 1001 125, 129, 137; RMSNorm, fp32 4096
// x 4096 32.4, 38.5, 39.9.  (Odd rows alone would do with 2; aligned ones decide.)
__host__ __device__ constexpr int cn_stages(int lanes, int teams, int nv, int V) {
    const int gamma = lanes * nv * V * 4, row = teams * ((lanes * nv + 1) * 16 + lanes * nv * V);
    return V == 8 && gamma + 3 * row <= 220 * 1024 ? 3 : 2;
}

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
    Extent ed;
};

template <int LPR, int TEAMS>
__device__ __forceinline__ void team_meets(int team) {
    if constexpr (LPR == 32)
        __syncwarp();
    else if constexpr (TEAMS == 1)
        __syncthreads();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(LPR) : "memory");
}

// The sum of W warps' values in shared memory.
template <int W>
__device__ __forceinline__ float warps_sum(const float* v) {
    float s = 0.f;
    if constexpr (W % 4 == 0) {
#pragma unroll
        for (int w = 0; w < W; w += 4) {
            const float4 f = *reinterpret_cast<const float4*>(v + w);
            s += (f.x + f.y) + (f.z + f.w);
        }
    } else {
#pragma unroll
        for (int w = 0; w < W; ++w) s += v[w];
    }
    return s;
}

// LPR lanes hold a row, NV vectors each (lane l: vectors l, l + LPR, ...); TEAMS rows at a time.  WHOLE: rows of
// whole vectors at vectors' distance.  Others come as the aligned chunks that they lie in, a lane's vector being in two
// that follow one another, one of them its neighbour's, so that the team meets before it reads them.
template <typename T, int LPR, int TEAMS, int NV, bool RMS, bool WHOLE>
__global__ void __launch_bounds__(LPR* TEAMS) ckpt_norm_kernel(const CnParams p) {
    constexpr int V = Io<T>::kVec, H = Pairs<T>::kPairs, W = LPR / 32, S = cn_stages(LPR, TEAMS, NV, V);
    constexpr int kThreads = LPR * TEAMS;
    constexpr int NS = RMS ? 1 : 2;
    // xhat stays in registers between a row's two passes where they have room beside the column sums; else the
    // integers are read again.
    constexpr bool KEEP = RMS || NV * V <= 24;
    // gamma in fp32 [cols], then dy [S][NV][threads] and the integers behind it; at the end, the teams'
    // column sums [TEAMS][NS][cols] in the place of the two.
    extern __shared__ __align__(16) float smem[];
    __shared__ __align__(16) float red[2][TEAMS][NS][W];
    const int tid = threadIdx.x, lane = tid & 31;
    const int team = tid / LPR, wt = (tid - team * LPR) / 32;
    const int cols = p.cols, blocks = ckpt_blocks(cols), padded = blocks * kCkptBlock;
    float* gamma = smem;
    float* fold = smem + padded;
    // Rows of dy as chunks, LPR NV and one more each; the integers, each lane's for itself.
    constexpr int kChunks = LPR * NV + 1;
    uint4* sd = reinterpret_cast<uint4*>(fold) + team * kChunks;
    unsigned char* sq = reinterpret_cast<unsigned char*>(fold) + (size_t)S * TEAMS * kChunks * 16 + tid * V;
    // (Pieces of a warp that follow one another where chunks between them are to be stored whole.)
    auto column = [&](int v) { return ((WHOLE ? v * LPR + wt * 32 : (wt * NV + v) * 32) + lane) * V; };
    const int step = (int)gridDim.x * TEAMS;  // (row + 2 steps stay below 2^31: LN_MAX_ROWS leaves room for them)
    const int row0 = (int)blockIdx.x * TEAMS + team;
    // Where this lane's first vector is, of the row to copy next and of the row to store next.
    const size_t lead = (size_t)(S - 1) * step;
    const T* next_dy = static_cast<const T*>(p.dy) + (size_t)row0 * cols + column(0);
    const int8_t* next_q = p.q + (size_t)row0 * padded + column(0);
    T* dx = static_cast<T*>(p.dx) + (size_t)row0 * cols;
    pdl_enter();
    auto issue = [&](int row, const T* dy, const int8_t* q, int stage) {
        if (row < p.rows) {
            uint4* to = sd + stage * (TEAMS * kChunks);
            if constexpr (WHOLE) {
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    if (column(v) < cols) copy_async<16>(to + column(v) / V, dy + (column(v) - column(0)));
            } else {
                const RowIn<T> in(dy - column(0), cols, p.ed);
                const int sh = (int)((unsigned)reinterpret_cast<uintptr_t>(in.row) & 15u) / (int)sizeof(T);
                const T* mine = in.row + (column(0) - sh);
                uint4* mine_to = to + column(0) / V;
                if (in.inside) {
#pragma unroll
                    for (int v = 0; v < NV; ++v)
                        if (column(v) - sh < cols) copy_async<16>(mine_to + v * 32, mine + v * 32 * V);
                } else {  // the tensor's first and last row
#pragma unroll 1
                    for (int v = 0; v < NV; ++v)
                        if (column(v) - sh < cols)
                            mine_to[v * 32] = chunk_at<T>(reinterpret_cast<const char*>(mine + v * 32 * V), p.ed);
                }
                if (tid - team * LPR == LPR - 1 && LPR * NV * V - sh < cols)
                    to[LPR * NV] = chunk_at<T>(reinterpret_cast<const char*>(in.row + (LPR * NV * V - sh)), p.ed);
            }
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (column(v) < cols) copy_async<V>(sq + (stage * NV + v) * (kThreads * V), q + (column(v) - column(0)));
        }
        copies_commit();
    };
#pragma unroll
    for (int s = 0; s < S - 1; ++s)
        issue(row0 + s * step, next_dy + (size_t)s * step * cols, next_q + (size_t)s * step * padded, s);
    // gamma's (and the column sums') groups of V: first halves, then second halves, so that 32 lanes read 512
    // consecutive bytes.
    auto place = [&](int c) { return ((c % V / 4) * (padded / V) + c / V) * 4 + c % 4; };
    for (int i = tid; i < padded; i += kThreads)
        gamma[place(i)] = i < cols ? Io<T>::to_f(static_cast<const T*>(p.gamma)[i]) : 0.f;
    f2 sg[NV][H], sb[RMS ? 1 : NV][H];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int h = 0; h < H; ++h) {
            sg[v][h] = f2_splat(0.f);
            if constexpr (!RMS) sb[v][h] = f2_splat(0.f);
        }
    __syncthreads();
    float mean_n = 0.f, rstd_n = 0.f;
    uint32_t kn[NV];
    auto scales = [&](int row) {
        if (row >= p.rows) return;
        rstd_n = load_ahead(p.rstd + row);
        if constexpr (!RMS) mean_n = load_ahead(p.mean + row);
        const uint8_t* k = p.k + (size_t)row * blocks;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (column(v) < cols) kn[v] = load_ahead(k + column(v) / kCkptBlock);
    };
    scales(row0);
    const float inv = 1.0f / (float)cols;
    int parity = 0, stage = 0;
    for (int row = row0; row < p.rows; row += step, parity ^= 1) {
        f2 x[KEEP ? NV : 1][H];
        // (Taken here, not where they were loaded: what is made of them would wait for the loads there.)
        float mean = mean_n, rstd = rstd_n;
        uint32_t kk[NV];
        asm volatile("" : "+f"(mean), "+f"(rstd));
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            kk[v] = kn[v];
            asm volatile("" : "+r"(kk[v]));
        }
        const f2 m2 = f2_splat(-mean), r2 = f2_splat(rstd);
        const unsigned s_row = WHOLE ? 0u : (unsigned)reinterpret_cast<uintptr_t>(next_dy - column(0)) & 15u;
        // A vector of dy, and of xhat.
        const uint4* chunks = sd + stage * (TEAMS * kChunks);
        auto load_dy = [&](int v, f2(&dy)[H]) {
            const int col = column(v);
            uint4 d = chunks[col / V];
            if constexpr (!WHOLE) {
                if (s_row != 0) d = join_at(d, chunks[col / V + 1], s_row);
                if (col + V > cols) d = first_of<T>(d, cols - col);
            }
            Pairs<T>::unpack(d, dy);
        };
        auto load_xhat = [&](int v, f2(&xv)[H]) {
            CkptRaw<T> raw;
            raw.k = kk[v];
            raw.take(sq + (stage * NV + v) * (kThreads * V));
            raw.values(xv, m2);
#pragma unroll
            for (int h = 0; h < H; ++h) xv[h] = f2_mul(xv[h], r2);
        };
        // gamma dy.
        auto times_gamma = [&](int v, const f2(&dy)[H], f2(&g)[H]) {
            const float4* gp = reinterpret_cast<const float4*>(gamma) + column(v) / V;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float4 g4 = gp[h / 2 * (padded / V)];
                g[h] = f2_mul(h & 1 ? f2_make(g4.z, g4.w) : f2_make(g4.x, g4.y), dy[h]);
            }
        };
        copies_wait<S - 2>();
        if constexpr (!WHOLE) team_meets<LPR, TEAMS>(team);
        f2 a = f2_splat(0.f), b = f2_splat(0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (column(v) >= cols) continue;
            f2 dy[H], g[H];
            f2(&xv)[H] = x[KEEP ? v : 0];
            load_dy(v, dy);
            load_xhat(v, xv);
            times_gamma(v, dy, g);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                sg[v][h] = f2_fma(dy[h], xv[h], sg[v][h]);
                if constexpr (!RMS) {
                    sb[v][h] = f2_add(sb[v][h], dy[h]);
                    a = f2_add(a, g[h]);
                }
                b = f2_fma(g[h], xv[h], b);
            }
        }
        issue(row + (S - 1) * step, next_dy + lead * cols, next_q + lead * padded, stage == 0 ? S - 1 : stage - 1);
        next_dy += (size_t)step * cols;
        next_q += (size_t)step * padded;
        scales(row + step);
        float sa = f2_lo(a) + f2_hi(a), sx = f2_lo(b) + f2_hi(b);
        if constexpr (RMS) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sx += __shfl_xor_sync(kFullMask, sx, o);
        } else {
            warp_sum2(sa, sx);
        }
        if constexpr (W > 1) {
            if (lane == 0) {
                red[parity][team][0][wt] = sx;
                if constexpr (!RMS) red[parity][team][NS - 1][wt] = sa;
            }
            team_meets<LPR, TEAMS>(team);
            sx = warps_sum<W>(red[parity][team][0]);
            if constexpr (!RMS) sa = warps_sum<W>(red[parity][team][NS - 1]);
        }
        const f2 a2 = f2_splat(-sa * inv), b2 = f2_splat(-sx * inv);
        RowOut<T, 32> out;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int col = column(v);
            if (col - lane * V >= cols) continue;  // the same in the whole warp
            uint4 u = make_uint4(0, 0, 0, 0);
            if (col < cols) {
                f2 dy[H], g[H];
                load_dy(v, dy);
                times_gamma(v, dy, g);
                if constexpr (!KEEP) load_xhat(v, x[0]);
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    if constexpr (!RMS) g[h] = f2_add(g[h], a2);
                    dy[h] = f2_mul(r2, f2_fma(x[KEEP ? v : 0][h], b2, g[h]));
                }
                u = Pairs<T>::pack(dy);
            }
            if constexpr (WHOLE) {
                if (col < cols) st_stream(dx + col, u);
            } else {
                out.put(dx, col, cols, u, v == 0, v == NV - 1);
            }
        }
        dx += (size_t)step * cols;
        if (++stage == S) stage = 0;
    }
    copies_wait<0>();
    // The block's column sums, its teams' in order.
    float* part = p.part + (size_t)blockIdx.x * NS * cols;
    __syncthreads();  // (no lane's copies are under way, or unread, any more)
    if constexpr (TEAMS > 1) {
        float4* mine = reinterpret_cast<float4*>(fold + (size_t)team * NS * padded);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int col = column(v);
            if (col >= padded) continue;
#pragma unroll
            for (int j = 0; j < V / 4; ++j) {
                const int at = j * (padded / V) + col / V;
                mine[at] = make_float4(f2_lo(sg[v][2 * j]), f2_hi(sg[v][2 * j]), f2_lo(sg[v][2 * j + 1]), f2_hi(sg[v][2 * j + 1]));
                if constexpr (!RMS)
                    mine[padded / 4 + at] =
                        make_float4(f2_lo(sb[v][2 * j]), f2_hi(sb[v][2 * j]), f2_lo(sb[v][2 * j + 1]), f2_hi(sb[v][2 * j + 1]));
            }
        }
        __syncthreads();
        for (int i = tid; i < NS * cols; i += kThreads) {
            const int st = !RMS && i >= cols, at = st * padded + place(i - st * cols);
            float s = fold[at];
#pragma unroll
            for (int t = 1; t < TEAMS; ++t) s += fold[(size_t)t * NS * padded + at];
            part[i] = s;
        }
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int col = column(v);
#pragma unroll
            for (int st = 0; st < NS; ++st) {
                const f2(&f)[H] = st ? sb[RMS ? 0 : v] : sg[v];
                if constexpr (WHOLE) {  // (rows of the partial sums start at 16 bytes)
                    if (col >= cols) continue;
#pragma unroll
                    for (int j = 0; j < V / 4; ++j)
                        *reinterpret_cast<float4*>(part + st * cols + col + 4 * j) =
                            make_float4(f2_lo(f[2 * j]), f2_hi(f[2 * j]), f2_lo(f[2 * j + 1]), f2_hi(f[2 * j + 1]));
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        if (col + e < cols) part[st * cols + col + e] = e & 1 ? f2_hi(f[e / 2]) : f2_lo(f[e / 2]);
                }
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
    int lanes, teams, nv;
};
// By capacity: lanes * nv vectors a row.  16 warps a block, one of which an SM holds: 128 registers a lane, and one
// row of partial sums an SM.  (Smaller blocks, by loads in time: bf16 8192 x 768 28 us for 12.5; a wide row
// by 16 warps, one at a time, for two teams of 8: 4096 x 8192 46 us for 38.)
constexpr CnShape kCnShapes[] = {{32, 16, 1}, {32, 16, 2}, {32, 16, 3}, {32, 16, 4}, {64, 8, 3}, {64, 8, 4},
                                 {128, 4, 3}, {128, 4, 4}, {256, 2, 3}, {256, 2, 4}, {512, 1, 3}, {512, 1, 4}, {512, 1, 8}};
constexpr int kCnCount = sizeof(kCnShapes) / sizeof(kCnShapes[0]);

template <typename T, bool RMS, bool WHOLE, int I>
const void* cn_kernel_of() {
    constexpr CnShape s = kCnShapes[I];
    if constexpr (s.nv == 8 && sizeof(T) == 2)
        return nullptr;  // LN_MAX_COLS in bf16 need no more than 4
    else
        return (const void*)ckpt_norm_kernel<T, s.lanes, s.teams, s.nv, RMS, WHOLE>;
}

template <typename T, bool RMS, bool WHOLE, int... I>
const void* cn_kernel(int shape, std::integer_sequence<int, I...>) {
    const void* found = nullptr;
    ((void)(shape == I && (found = cn_kernel_of<T, RMS, WHOLE, I>())), ...);
    return found;
}

// Blocks of any shape resident on an SM at most.
constexpr int kCnMaxPerSm = 4;

template <typename T, bool RMS>
cudaError_t launch_cn_t(const CkptNormArgs& a, cudaStream_t stream, int* launches) {
    constexpr int V = Io<T>::kVec;
    *launches = 0;
    const int nvec = (a.cols + V - 1) / V;
    int shape = 0;
    while (shape < kCnCount && kCnShapes[shape].lanes * kCnShapes[shape].nv < nvec) ++shape;
    if (shape == kCnCount) return cudaErrorInvalidValue;
    const CnShape& sh = kCnShapes[shape];
    auto aligned = [](const void* t) { return (reinterpret_cast<uintptr_t>(t) & 15u) == 0; };
    const bool whole = aligned(a.dy) && aligned(a.dx) && a.cols % V == 0;
    constexpr auto all = std::make_integer_sequence<int, kCnCount>();
    const void* kern = whole ? cn_kernel<T, RMS, true>(shape, all) : cn_kernel<T, RMS, false>(shape, all);
    if (!kern) return cudaErrorInvalidValue;
    const int threads = sh.lanes * sh.teams;
    int stats = RMS ? 1 : 2;
    const size_t staged = (size_t)cn_stages(sh.lanes, sh.teams, sh.nv, V) *
                          ((size_t)sh.teams * (sh.lanes * sh.nv + 1) * 16 + (size_t)sh.nv * threads * V);
    const size_t folded = sh.teams > 1 ? (size_t)sh.teams * stats * ckpt_blocks(a.cols) * kCkptBlock * sizeof(float) : 0;
    const size_t smem = (size_t)ckpt_blocks(a.cols) * kCkptBlock * sizeof(float) + std::max(staged, folded);
    cudaError_t e = smem > 40 * 1024 ? allow_smem(kern, smem) : cudaSuccess;
    if (e != cudaSuccess) return e;
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
    const int per_sm = std::min(kCnMaxPerSm, std::max(1, blocks_per_sm(kern, threads, smem)));
    int blocks = std::min(per_sm * device_info(-1).sms, (a.rows + sh.teams - 1) / sh.teams);
    void* args[] = {&p};
    e = launch_kernel(kern, dim3(blocks), dim3(threads), smem, stream, args, false);
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
