// ckpt8_norm.cu -- the LayerNorm's and RMSNorm's backward from an input kept in 8 bits.
//
// With x as the checkpoint gives it back, xhat = (x - mean) rstd (RMSNorm: mean 0) and g = gamma dy:
//   dx = rstd (g - (sum g + xhat sum g xhat) / cols)        (RMSNorm: without the first sum)
//   dgamma = sum over rows of dy xhat,  dbeta = sum over rows of dy
// ("Accelerating Transformer on GPU (II): Training with LightSeq2", section 2.1; mean and rstd are the
// forward's, of the input itself).  A row is held in registers by 1 to 32 warps (a team), at 8 to 24 columns a lane,
// and each lane keeps the column sums of its columns over all rows that its team takes.  dy and the integers of
// the next 2 or 3 rows are on their way meanwhile, by asynchronous copies of 16 and 8 (4) bytes into
// shared memory that each lane makes and reads for itself, without barriers.  A block adds its teams' column sums in
// order and leaves one row of partial sums for each statistic; a second, dependent launch adds those of a column,
// 32 interleaved groups and then the groups, with their rounding errors carried along.  No atomics: results are the
// same from run to run.
#include <algorithm>
#include <utility>

#include "ckpt8.cuh"
#include "ln_finish.cuh"
#include "rel_ops.h"
#include "row_io.cuh"

namespace lnk {
namespace {

// Rows of a team in shared memory or on their way there.
__host__ __device__ constexpr int cn_stages(int lanes, int nv) { return lanes == 512 && nv == 4 ? 3 : 4; }

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

template <int BYTES>
__device__ __forceinline__ void copy_async(void* to, const void* from) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_addr(to)), "l"(from), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Loads that stay where they are written, an iteration before their use.
__device__ __forceinline__ float load_ahead(const float* p) {
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t load_ahead(const uint8_t* p) {
    uint32_t v;
    asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// The sum of W warps' values in shared memory, in order.
template <int W>
__device__ __forceinline__ float warps_sum(const float* v) {
    float s = 0.f;
    if constexpr (W % 4 == 0) {
#pragma unroll
        for (int w = 0; w < W; w += 4) {
            const float4 f = *reinterpret_cast<const float4*>(v + w);
            s += f.x;
            s += f.y;
            s += f.z;
            s += f.w;
        }
    } else {
#pragma unroll
        for (int w = 0; w < W; ++w) s += v[w];
    }
    return s;
}

// LPR lanes hold a row, NV vectors each (lane l: vectors l, l + LPR, ...); TEAMS rows at a time.  WHOLE: rows of
// whole vectors at vectors' distance; others are loaded when they are needed.
template <typename T, int LPR, int TEAMS, int NV, bool RMS, bool WHOLE>
__global__ void __launch_bounds__(LPR* TEAMS) ckpt_norm_kernel(const CnParams p) {
    constexpr int V = Io<T>::kVec, H = Pairs<T>::kPairs, W = LPR / 32, S = cn_stages(LPR, NV);
    constexpr int kThreads = LPR * TEAMS;
    constexpr int NS = RMS ? 1 : 2;
    // gamma in fp32 [cols], then dy [S][NV][threads] and the integers behind it; at the end, the teams'
    // column sums [TEAMS][NS][cols] in the place of the two.
    extern __shared__ __align__(16) float smem[];
    __shared__ __align__(16) float red[2][TEAMS][NS][W];
    const int tid = threadIdx.x, lane = tid & 31;
    const int team = tid / LPR, wt = (tid - team * LPR) / 32;
    const int cols = p.cols, blocks = ckpt_blocks(cols), padded = blocks * kCkptBlock;
    float* gamma = smem;
    float* fold = smem + padded;
    uint4* sd = reinterpret_cast<uint4*>(fold) + tid;
    unsigned char* sq = reinterpret_cast<unsigned char*>(fold) + (size_t)S * NV * kThreads * 16 + tid * V;
    auto column = [&](int v) { return (v * LPR + wt * 32 + lane) * V; };
    const int step = (int)gridDim.x * TEAMS;  // (row + 2 steps stay below 2^31: LN_MAX_ROWS leaves room for them)
    const int row0 = (int)blockIdx.x * TEAMS + team;
    // Where this lane's first vector is, of the row to copy next and of the row to store next.
    const size_t lead = (size_t)(S - 1) * step;
    const T* next_dy = static_cast<const T*>(p.dy) + (size_t)row0 * cols + column(0);
    const int8_t* next_q = p.q + (size_t)row0 * padded + column(0);
    T* dx = static_cast<T*>(p.dx) + (size_t)row0 * cols;
    pdl_enter();
    auto issue = [&](int row, const T* dy, const int8_t* q, int stage) {
        if constexpr (WHOLE) {
            if (row < p.rows) {
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    if (column(v) < cols) {
                        copy_async<16>(sd + (stage * NV + v) * kThreads, dy + v * LPR * V);
                        copy_async<V>(sq + (stage * NV + v) * (kThreads * V), q + v * LPR * V);
                    }
            }
            copies_commit();
        }
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
        uint4 d[NV];
        f2 x[NV][H];
        // (Taken here, not where they were loaded: what is made of them would wait for the loads there.)
        float mean = mean_n, rstd = rstd_n;
        asm volatile("" : "+f"(mean), "+f"(rstd));
        const f2 m2 = f2_splat(-mean), r2 = f2_splat(rstd);
        copies_wait<S - 2>();
        f2 a = f2_splat(0.f), b = f2_splat(0.f);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int col = column(v);
            if (col >= cols) continue;
            CkptRaw<T> raw;
            raw.k = kn[v];
            asm volatile("" : "+r"(raw.k));
            if constexpr (WHOLE) {
                d[v] = sd[(stage * NV + v) * kThreads];
                raw.take(sq + (stage * NV + v) * (kThreads * V));
            } else {
                const T* dy = next_dy - column(0);
                d[v] = load_columns<T>(RowIn<T>(dy, cols, p.ed), col, cols, p.ed);
                if (col + V > cols) d[v] = first_of<T>(d[v], cols - col);
                raw.take(next_q + (col - column(0)));
            }
            raw.values(x[v], m2);
            f2 dy[H];
            Pairs<T>::unpack(d[v], dy);
            const float4* gp = reinterpret_cast<const float4*>(gamma) + col / V;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float4 g4 = gp[h / 2 * (padded / V)];
                const f2 g = f2_mul(h & 1 ? f2_make(g4.z, g4.w) : f2_make(g4.x, g4.y), dy[h]);
                x[v][h] = f2_mul(x[v][h], r2);
                sg[v][h] = f2_fma(dy[h], x[v][h], sg[v][h]);
                if constexpr (!RMS) {
                    sb[v][h] = f2_add(sb[v][h], dy[h]);
                    a = f2_add(a, g);
                }
                b = f2_fma(g, x[v][h], b);
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
            if constexpr (TEAMS == 1)
                __syncthreads();
            else
                asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(LPR) : "memory");
            sx = warps_sum<W>(red[parity][team][0]);
            if constexpr (!RMS) sa = warps_sum<W>(red[parity][team][NS - 1]);
        }
        const f2 a2 = f2_splat(-sa * inv), b2 = f2_splat(-sx * inv);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int col = column(v);
            if (col - lane * V >= cols) continue;  // the same in the whole warp
            uint4 u = make_uint4(0, 0, 0, 0);
            if (col < cols) {
                f2 dy[H];
                Pairs<T>::unpack(d[v], dy);
                const float4* gp = reinterpret_cast<const float4*>(gamma) + col / V;
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const float4 g4 = gp[h / 2 * (padded / V)];
                    f2 g = f2_mul(h & 1 ? f2_make(g4.z, g4.w) : f2_make(g4.x, g4.y), dy[h]);
                    if constexpr (!RMS) g = f2_add(g, a2);
                    dy[h] = f2_mul(r2, f2_fma(x[v][h], b2, g));
                }
                u = Pairs<T>::pack(dy);
            }
            if constexpr (WHOLE) {
                if (col < cols) st_stream(dx + col, u);
            } else {
                store_columns<T>(dx, col, cols, u);
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
// By capacity: lanes * nv vectors a row.  16 warps a block, so that an SM leaves one row of partial sums or two;
// a lane's sums, x and dy of 24 columns in bf16 fill 128 registers, of 32 where there is one statistic.
constexpr CnShape kCnShapes[] = {{32, 16, 1}, {32, 16, 2}, {32, 16, 3}, {32, 16, 4}, {64, 8, 2}, {64, 8, 3}, {64, 8, 4},
                                 {128, 4, 2}, {128, 4, 3}, {128, 4, 4}, {256, 2, 2}, {256, 2, 3}, {256, 2, 4},
                                 {512, 1, 2}, {512, 1, 3}, {512, 1, 4}, {1024, 1, 4}};
constexpr int kCnCount = sizeof(kCnShapes) / sizeof(kCnShapes[0]);

// Whether a shape is used: of those with 4 vectors a lane, the widest, and any that 128 registers hold.
constexpr bool cn_fits(const CnShape& s, bool rms, bool f32) {
    return s.lanes == 256 && s.nv == 4 ? f32 : s.nv < 4 || s.lanes >= 512 || rms || f32;
}

template <typename T, bool RMS, bool WHOLE, int I>
const void* cn_kernel_of() {
    constexpr CnShape s = kCnShapes[I];
    if constexpr (s.lanes == 1024 && (sizeof(T) == 2 || WHOLE))
        return nullptr;  // 512 lanes hold LN_MAX_COLS in bf16; fp32's rows do not fit the stages
    else if constexpr (!cn_fits(s, RMS, sizeof(T) == 4))
        return nullptr;
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
    while (shape < kCnCount && (kCnShapes[shape].lanes * kCnShapes[shape].nv < nvec ||
                                !cn_fits(kCnShapes[shape], RMS, sizeof(T) == 4)))
        ++shape;
    if (shape == kCnCount) return cudaErrorInvalidValue;
    const CnShape& sh = kCnShapes[shape];
    auto aligned = [](const void* t) { return (reinterpret_cast<uintptr_t>(t) & 15u) == 0; };
    const bool whole = aligned(a.dy) && aligned(a.dx) && a.cols % V == 0 && sh.lanes < 1024;
    constexpr auto all = std::make_integer_sequence<int, kCnCount>();
    const void* kern = whole ? cn_kernel<T, RMS, true>(shape, all) : cn_kernel<T, RMS, false>(shape, all);
    if (!kern) return cudaErrorInvalidValue;
    const int threads = sh.lanes * sh.teams;
    int stats = RMS ? 1 : 2;
    const size_t staged = whole ? (size_t)cn_stages(sh.lanes, sh.nv) * sh.nv * threads * (16 + V) : 0;
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
