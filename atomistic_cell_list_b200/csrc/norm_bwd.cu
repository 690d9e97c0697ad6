// Layer norm of irreducible features: backward (the mathematics and the layout are in norm.cuh).
#include "launch.cuh"
#include "norm.cuh"

namespace e2f {
namespace {

constexpr int kBwdWarps = 4;  // of a block, at 255 registers: x and grad_y of a unit
constexpr int kStatNodes = 72;  // most nodes of a unit: 9 for each of 8 teams
constexpr int kStatBytes = 8 * kStatNodes;

// The units of degree l that this block takes. Each lane keeps the weight
// gradient of its channels in registers until the end, then the block's lanes
// that share channels are added in order: no atomics. part: [block][C], then
// [block of degree 0][C] for the bias. x and grad_y of a unit stay in registers
// between the sums and the gradient: 30,000 atoms, L = 4, C = 128, fp32 with a skip
// gradient, 1.54 GB in 248 us (6.2 TB/s); 10,027 atoms, C = 64, bf16, 161 MB in 36 us.
// Two vectors a lane (C above 128), 12,000 atoms, L = 4, C = 256: fp32 with a skip gradient
// 1.23 GB in 211 us, bf16 769 MB in 197 us, codes with a skip gradient 1.0 GB in 470 us.
template <int XT, int NI, int l>
__device__ __forceinline__ void norm_bwd_degree(const NormBwdArgs& a, int TL, const Slots& sl, char* smem) {
    using U = Unit<NI, l>;
    constexpr int V = 4, E = vec_bytes<XT>() / 4, R = U::R, B = U::B;
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, lane = threadIdx.x & 31, t = lane & (TL - 1), C = a.C;
    const int K = (a.L + 1) * (a.L + 1), teams = 32 / TL, team = lane / TL, team0 = team * (B * R);
    const uint32_t smem_s = (uint32_t)__cvta_generic_to_shared(smem);
    const uint32_t zeros = smem_s + warps * sl.stages * sl.stage_bytes;
    const uint32_t mine_s = smem_s + warp * sl.stages * sl.stage_bytes;
    int c[NI];
    bool in[NI];
    float w[NI][V], dw[NI][V] = {}, db[NI][V] = {};
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        in[i] = (t + TL * i) * V < C;
        c[i] = in[i] ? (t + TL * i) * V : 0;
        load_vec<kF32, V>(a.w, l * C + c[i], w[i]);
    }
    const int blocks = sl.at[l + 1] - sl.at[l];
    const int64_t step = (int64_t)blocks * warps, units = (a.n + B * teams - 1) / (B * teams);
    int64_t k = (int)blockIdx.x - sl.at[l] + (int64_t)blocks * warp;
    auto fetch = [&](int64_t k, int stage) {
        if (k < units) {
            const U u(k, a.n, K, TL);
            uint32_t to = mine_s + stage * sl.stage_bytes;
            u.template fetch<XT>(a.x, C, K, TL, to);
            u.template fetch<kF32>(a.gy, C, K, TL, to + sl.o1);
            if (a.skip) u.template fetch<kF32>(a.skip, C, K, TL, to + sl.o2);
            to += sl.o3 + 4 * team * B;  // statistics: [team][node] rstd, then mean
            for (int b = t; b < u.have; b += TL) {
                const int64_t node = u.first + b * teams;
                cp_async_small<4>(to + 4 * b, a.rstd + node * (a.L + 1) + l);
                if (l == 0) cp_async_small<4>(to + 4 * (kStatNodes + b), a.mean + node);
            }
        }
        cp_commit();
    };
    uint32_t scale[B * R][NI] = {};  // of the next unit, where x has any
    if (XT == kMXI8 && k < units) U(k, a.n, K, TL).scales(a.xs, a.nb, K, TL, c, scale);
    for (int s = 0; s + 1 < sl.stages; ++s) fetch(k + s * step, s);
    for (int s = 0; k < units; k += step, s = s + 1 == sl.stages ? 0 : s + 1) {
        const U u(k, a.n, K, TL);
        __syncwarp();  // the whole warp is done with the stage that is filled next
        fetch(k + (sl.stages - 1) * step, s == 0 ? sl.stages - 1 : s - 1);
        cp_wait(sl.stages - 1);
        __syncwarp();
        const uint32_t st = mine_s + s * sl.stage_bytes;
        const float* stat = reinterpret_cast<const float*>(smem + (st - smem_s) + sl.o3) + team * B;
        const float* mean[NI];  // of lanes beyond the row: zero, for (0 - mean) rstd may be infinite and 0 times it NaN
#pragma unroll
        for (int i = 0; i < NI; ++i)
            mean[i] = in[i] ? stat + kStatNodes : reinterpret_cast<const float*>(smem + (zeros - smem_s));
        float x[B][R][NI][V], g[B][R][NI][V], r[B], s1[B], s2[B];  // x becomes xh, g becomes u = grad_y weight
        float uw[NI][V] = {}, ub[NI][V] = {};  // the unit's part of dw and db, so that the chains of additions stay short
#pragma unroll
        for (int b = 0; b < B; ++b) {
            r[b] = stat[b];
            s1[b] = s2[b] = 0.f;
            const bool ok = b < u.have;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                // lanes beyond the row: zero, not (0 - mean) rstd, which may be infinite
                const float mu = l == 0 ? mean[i][b] : 0.f;
                const uint32_t p = in[i] ? st + (team0 * C + c[i]) * E : zeros;
                const uint32_t pg = in[i] ? st + sl.o1 + (team0 * C + c[i]) * 4 : zeros;
                const int pitch = in[i] ? C : 0;
#pragma unroll
                for (int m = 0; m < R; ++m) {
                    float (&xv)[V] = x[b][m][i];
                    Raw4<XT> raw;
                    raw.from(p + (b * R + m) * pitch * E);
                    if constexpr (XT == kMXI8) raw.s = scale[b * R + m][i];
                    raw.get(xv);
                    Raw4<kF32> e;
                    e.from(pg + (b * R + m) * pitch * 4);
                    const float gv[V] = {e.a.x, e.a.y, e.a.z, e.a.w};
                    for (int k = 0; k < V; ++k) {
                        const float xh = (l == 0 ? xv[k] - mu : xv[k]) * r[b], uk = gv[k] * w[i][k];
                        if (ok) uw[i][k] += gv[k] * xh;
                        s2[b] += uk * xh;
                        if constexpr (l == 0) {
                            if (ok) ub[i][k] += gv[k];
                            s1[b] += uk;
                        }
                        xv[k] = xh;
                        g[b][m][i][k] = uk;
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NI; ++i)
            for (int k = 0; k < V; ++k) {
                dw[i][k] += uw[i][k];
                if constexpr (l == 0) db[i][k] += ub[i][k];
            }
        if constexpr (XT == kMXI8)
            if (k + step < units) U(k + step, a.n, K, TL).scales(a.xs, a.nb, K, TL, c, scale);
        if constexpr (l == 0) team_sum(s1, TL);
        team_sum(s2, TL);
        const int64_t base = u.row0 * C;
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const float m1 = s1[b] * a.inv_c * r[b], m2 = s2[b] * (a.inv_c * (1.f / R)) * r[b];
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                float* to = a.gx + base + (int64_t)(b * teams * K) * C + c[i];
                if (b < u.have && in[i])
#pragma unroll
                    for (int m = 0; m < R; ++m) {
                        float o[V];
                        for (int k = 0; k < V; ++k)
                            o[k] = fmaf(-x[b][m][i][k], m2, l == 0 ? fmaf(r[b], g[b][m][i][k], -m1) : r[b] * g[b][m][i][k]);
                        if (a.skip) {
                            Raw4<kF32> e;
                            e.from(st + sl.o2 + ((team0 + b * R + m) * C + c[i]) * 4);
                            o[0] += e.a.x; o[1] += e.a.y; o[2] += e.a.z; o[3] += e.a.w;
                        }
                        store_vec<kF32, V>(to, 0, o);
                        to += C;
                    }
            }
        }
    }
    if (!a.part) return;
    float* sh = reinterpret_cast<float*>(smem);  // the stages, free now: [warps][32 lanes][NI][V]
#pragma unroll
    for (int pass = 0; pass < (l == 0 ? 2 : 1); ++pass) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NI; ++i)
            for (int k = 0; k < V; ++k) sh[((warp * 32 + lane) * NI + i) * V + k] = pass == 0 ? dw[i][k] : db[i][k];
        __syncthreads();
        float* out = a.part + (int64_t)(blockIdx.x + (pass == 0 ? 0 : sl.at[kMaxL + 1])) * C;
        for (int o = threadIdx.x; o < C; o += blockDim.x) {
            const int vec = o / V, i = vec / TL, tt = vec % TL;
            float sum = 0.f;
            for (int q = 0; q < warps * teams; ++q) sum += sh[((q * TL + tt) * NI + i) * V + o % V];
            out[o] = sum;
        }
    }
}

template <int XT, int NI>
__global__ void __launch_bounds__(32 * kBwdWarps, 2) k_norm_bwd_teams(NormBwdArgs a, int TL, Slots sl) {
    extern __shared__ __align__(16) char smem[];
    if (threadIdx.x < 16)
        reinterpret_cast<float*>(smem + (blockDim.x >> 5) * sl.stages * sl.stage_bytes)[threadIdx.x] = 0.f;
    __syncthreads();
    const int blk = blockIdx.x;
    if (blk < sl.at[1]) norm_bwd_degree<XT, NI, 0>(a, TL, sl, smem);
    else if (blk < sl.at[2]) norm_bwd_degree<XT, NI, 1>(a, TL, sl, smem);
    else if (blk < sl.at[3]) norm_bwd_degree<XT, NI, 2>(a, TL, sl, smem);
    else if (blk < sl.at[4]) norm_bwd_degree<XT, NI, 3>(a, TL, sl, smem);
    else norm_bwd_degree<XT, NI, 4>(a, TL, sl, smem);
}

// One block per (node, degree), the blocks split over the degrees as the rows
// are: degree l has blocks [g l^2, g (l+1)^2). Each thread owns its channels,
// so the block's part of the weight gradient is summed in shared memory
// without atomics, in a fixed order. What the other kernels do not take (more than
// 256 channels at L >= 1, rows beyond what a block holds); it reads twice: 4,000 atoms,
// L = 4, C = 260, fp32 with a skip gradient, 416 MB in 378 us.
template <int XT, int V>
__global__ void k_norm_bwd_rows(NormBwdArgs a) {
    extern __shared__ float acc[];  // [C] weight, then [C] bias (l = 0)
    __shared__ float sh[32];
    const int K = (a.L + 1) * (a.L + 1), T = blockDim.x;
    int l = 0;
    while ((int)blockIdx.x >= a.g * (l + 1) * (l + 1)) ++l;
    const int rows = 2 * l + 1, nblk = a.g * rows;
    if (a.part)
        for (int c = threadIdx.x * V; c < a.C; c += T * V)
            for (int k = 0; k < V; ++k) {
                acc[c + k] = 0.f;
                if (l == 0) acc[a.C + c + k] = 0.f;
            }
    for (int64_t node = blockIdx.x - a.g * l * l; node < a.n; node += nblk) {
        const int64_t row0 = node * K + l * l;
        const float mu = l == 0 ? a.mean[node] : 0.f, r = a.rstd[node * (a.L + 1) + l];
        float s1 = 0.f, s2 = 0.f;
        for (int c = threadIdx.x * V; c < a.C; c += T * V) {
            float w[V];
            load_vec<kF32, V>(a.w, (int64_t)l * a.C + c, w);
            for (int m = 0; m < rows; ++m) {
                float x[V], g[V];
                load_feat<XT, V>(a.x, a.xs, row0 + m, a.C, a.nb, c, x);
                load_vec<kF32, V>(a.gy, (row0 + m) * a.C + c, g);
                for (int k = 0; k < V; ++k) {
                    const float xh = (x[k] - mu) * r, gx = g[k] * xh;
                    s1 += g[k] * w[k];
                    s2 += gx * w[k];
                    if (a.part) {
                        acc[c + k] += gx;
                        if (l == 0) acc[a.C + c + k] += g[k];
                    }
                }
            }
        }
        s1 = l == 0 ? block_sum(s1, sh) / a.C : 0.f;
        s2 = block_sum(s2, sh) / ((float)rows * a.C);
        for (int c = threadIdx.x * V; c < a.C; c += T * V) {
            float w[V];
            load_vec<kF32, V>(a.w, (int64_t)l * a.C + c, w);
            for (int m = 0; m < rows; ++m) {
                float x[V], g[V];
                load_feat<XT, V>(a.x, a.xs, row0 + m, a.C, a.nb, c, x);
                load_vec<kF32, V>(a.gy, (row0 + m) * a.C + c, g);
                float d[V];
                for (int k = 0; k < V; ++k) d[k] = r * (g[k] * w[k] - s1 - (x[k] - mu) * r * s2);
                if (a.skip) {
                    load_vec<kF32, V>(a.skip, (row0 + m) * a.C + c, g);
                    for (int k = 0; k < V; ++k) d[k] += g[k];
                }
                store_vec<kF32, V>(a.gx, (row0 + m) * a.C + c, d);
            }
        }
    }
    if (!a.part) return;
    for (int c = threadIdx.x * V; c < a.C; c += T * V)
        for (int k = 0; k < V; ++k) {
            a.part[(int64_t)blockIdx.x * a.C + c + k] = acc[c + k];
            if (l == 0) a.part[(int64_t)(a.g * K + blockIdx.x) * a.C + c + k] = acc[a.C + c + k];
        }
}

// L = 0: persistent blocks, one row at a time in registers, NV vectors of V values
// of x and of grad_y a thread, with the weight and bias gradient of its channels:
// each value is read once, and a row's loads are issued before the sums of the row
// before it. 8,192 rows of 4,096 fp32 values with a skip gradient: 537 MB in 101 us
// (5.3 TB/s; 113 us without the early loads). 20,000 rows of 1,001, value by value:
// 54 us; 4,096 rows of 5,001 with bf16 x: 79 us, bound by instructions.
// part: [block][C], then [block][C] for the bias.
template <int XT, int V, int NV, int TT>
__global__ void __launch_bounds__(TT ? TT : 1024) k_norm_bwd_held(NormBwdArgs a) {
    __shared__ float sh[2][32];
    const int T = TT ? TT : blockDim.x, C = a.C - threadIdx.x * V;  // this thread's vector j exists: j T V < C
    float dw[NV][V] = {}, db[NV][V] = {};
    const float* wp = a.w + threadIdx.x * V;
    float x[NV][V], g[NV][V], mu = 0.f, r = 0.f;
    auto load = [&](int64_t row, float (&x)[NV][V], float (&g)[NV][V], float& mu, float& r) {
        const int64_t base = row * a.C + threadIdx.x * V;
        const char* xp = static_cast<const char*>(a.x) + base * (vec_bytes<XT>() / 4);
        const float* gp = a.gy + base;
        mu = a.mean[row];
        r = a.rstd[row];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            for (int k = 0; k < V; ++k) x[j][k] = g[j][k] = 0.f;
            if (j * T * V < C) {
                if constexpr (XT == kMXI8)
                    load_codes<V>(static_cast<const int8_t*>(a.x), a.xs, row, a.C, a.nb, (j * T + threadIdx.x) * V, x[j]);
                else
                    load_vec<XT, V>(xp, j * T * V, x[j]);
                load_vec<kF32, V>(gp, j * T * V, g[j]);
            }
        }
    };
    if (blockIdx.x < a.n) load(blockIdx.x, x, g, mu, r);
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
        const int64_t base = row * a.C + threadIdx.x * V;
        const float* kp = a.skip + base;
        float* op = a.gx + base;
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * T * V < C) {
                float w[V];
                load_vec<kF32, V>(wp, j * T * V, w);
                for (int k = 0; k < V; ++k) {
                    const float xh = (x[j][k] - mu) * r, u = g[j][k] * w[k];
                    dw[j][k] += g[j][k] * xh;
                    db[j][k] += g[j][k];
                    s1 += u;
                    s2 += u * xh;
                    x[j][k] = xh;
                    g[j][k] = u;
                }
            }
        // the next row is on its way while this one's sums are formed
        float xn[NV][V], gn[NV][V], mun = 0.f, rn = 0.f;
        if (row + gridDim.x < a.n) load(row + gridDim.x, xn, gn, mun, rn);
        const float m1 = block_sum(s1, sh[0]) * a.inv_c, m2 = block_sum(s2, sh[1]) * a.inv_c;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * T * V < C) {
                float e[V] = {};
                if (a.skip) load_vec<kF32, V>(kp, j * T * V, e);
                for (int k = 0; k < V; ++k) e[k] += r * (g[j][k] - m1 - x[j][k] * m2);
                store_vec<kF32, V>(op, j * T * V, e);
            }
#pragma unroll
        for (int j = 0; j < NV; ++j)
            for (int k = 0; k < V; ++k) {
                x[j][k] = xn[j][k];
                g[j][k] = gn[j][k];
            }
        mu = mun;
        r = rn;
    }
    if (!a.part) return;
    float* part = a.part + (int64_t)blockIdx.x * a.C + threadIdx.x * V;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (j * T * V < C) {
            store_vec<kF32, V>(part, j * T * V, dw[j]);
            store_vec<kF32, V>(part + (int64_t)gridDim.x * a.C, j * T * V, db[j]);
        }
}

// Where the blocks' partials lie: `count` rows of `stride` values for each degree and the bias.
struct JoinPlan {
    int64_t base[kMaxL + 2], stride;
    int count[kMaxL + 2];
};

// Sums the partials. 32 warps share the rows of one column block, so that a few loads each
// are in flight at once: about 4 us for 296 blocks of 128 channels behind the first kernel,
// 6.9 us alone with cold caches.
__global__ void __launch_bounds__(1024) k_norm_join(const float* part, int L, int C, JoinPlan p, float* gw, float* gb) {
    __shared__ float sh[32][33];
    const int l = blockIdx.y, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, w = threadIdx.x >> 5;
    float* out = l <= L ? gw : gb;
    after_previous();
    if (!out) return;
    const float* q = part + p.base[l] + c;
    float s = 0.f;
    if (c < C)
#pragma unroll 10
        for (int r = w; r < p.count[l]; r += 32) s += q[r * p.stride];
    sh[w][lane] = s;
    __syncthreads();
    s = sh[lane][w];  // warp w sums column w
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int cw = blockIdx.x * 32 + w;
    if (lane == 0 && cw < C) out[(l <= L ? (int64_t)l * C : 0) + cw] = s;
}

template <int XT, int V>
cudaError_t launch_bwd_rows(const NormBwdArgs& a, cudaStream_t s) {
    const size_t smem = a.part ? 8 * (size_t)a.C : 0;
    if (smem > 40 * 1024) {  // without it a launch has 48 KB, the kernel's static 128 bytes among them
        cudaError_t e = cudaFuncSetAttribute(k_norm_bwd_rows<XT, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             8 * kMaxNormC);
        if (e != cudaSuccess) return e;
    }
    k_norm_bwd_rows<XT, V><<<a.g * (a.L + 1) * (a.L + 1), row_threads(a.C, V), smem, s>>>(a);
    return cudaGetLastError();
}

template <int XT, int NI>
cudaError_t launch_bwd_teams(const NormBwdArgs& a, const TeamPlan& p, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(k_norm_bwd_teams<XT, NI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kBlockSmem);
    if (e != cudaSuccess) return e;
    const int row = kUnitRows * NI * 32, o1 = row * vec_bytes<XT>(), o2 = o1 + row * 16;
    Slots sl{p.stage_bytes, p.stages, o1, o2, o2 + (a.skip ? row * 16 : 0), {}};
    std::copy(p.at, p.at + kMaxL + 2, sl.at);
    k_norm_bwd_teams<XT, NI><<<p.at[kMaxL + 1], 32 * p.warps, p.smem, s>>>(a, p.TL, sl);
    return cudaGetLastError();
}

// threads of k_norm_bwd_held, 0: not for this shape
int bwd_held(int L, int C) {
    if (L) return 0;
    if (C % 4 == 0) return held_threads(C, 4, 2);
    return C <= 1024 ? 128 : C <= 6144 ? 512 : 0;
}

// blocks of k_norm_bwd_held (what fits at once by registers: 1,024 threads of 64, at most 5 blocks, and one block of
// 512 threads of 128, value by value; a second wave costs more than it hides: 4,096 rows of 5,001 bf16 values 79 us
// in 148 blocks, 85 us in 296), or blocks per row of features of k_norm_bwd_rows
int rows_blocks(int64_t n, int L, int C) {
    const int t = bwd_held(L, C), threads = t == 512 && C % 4 ? 512 : 1024;
    const int most = t ? kSMs * std::max(1, std::min(5, threads / t)) : kNormBlocks / ((L + 1) * (L + 1));
    return (int)std::max<int64_t>(1, std::min<int64_t>(n, most));
}

template <int XT>
cudaError_t launch_bwd(NormBwdArgs a, float* gw, float* gb, cudaStream_t s) {
    const int K = (a.L + 1) * (a.L + 1);
    JoinPlan j{};
    cudaError_t e;
    auto join_degrees = [&](const int* at) {  // blocks of one degree, then the bias of those of degree 0
        j.stride = a.C;
        for (int l = 0; l < a.L + 2; ++l) {
            j.base[l] = (int64_t)(l <= a.L ? at[l] : at[kMaxL + 1]) * a.C;
            j.count[l] = l <= a.L ? at[l + 1] - at[l] : at[1];
        }
    };
    count_launch();
    if (use_teams(a.C)) {
        const TeamPlan p = team_plan(a.n, a.L, a.C, vec_bytes<XT>() + (a.skip ? 32 : 16), vec_bytes<XT>() + 32,
                                     kStatBytes, kBwdWarps);
        e = p.NI == 1 ? launch_bwd_teams<XT, 1>(a, p, s) : launch_bwd_teams<XT, 2>(a, p, s);
        join_degrees(p.at);
    } else if (a.C <= kTeamC) {
        int at[kMaxL + 2];
        e = run_norm_bwd_scalar(a, XT, at, s);
        join_degrees(at);
    } else {
        a.g = rows_blocks(a.n, a.L, a.C);
        if (const int t = bwd_held(a.L, a.C)) {
            if (a.C % 4 == 0) k_norm_bwd_held<XT, 4, 2, 0><<<a.g, t, 0, s>>>(a);
            else if (t == 128) k_norm_bwd_held<XT, 1, 8, 128><<<a.g, t, 0, s>>>(a);
            else k_norm_bwd_held<XT, 1, 12, 512><<<a.g, t, 0, s>>>(a);
            e = cudaGetLastError();
        } else
            e = a.C % 4 == 0 ? launch_bwd_rows<XT, 4>(a, s) : launch_bwd_rows<XT, 1>(a, s);
        j.stride = a.C;
        for (int l = 0; l < a.L + 2; ++l) {
            j.base[l] = (int64_t)a.g * (l <= a.L ? l * l : K) * a.C;
            j.count[l] = a.g * (l <= a.L ? 2 * l + 1 : 1);
        }
    }
    if (e != cudaSuccess || !a.part) return e;
    return launch_after(k_norm_join, dim3((a.C + 31) / 32, a.L + 2), 1024, 0, s, a.part, a.L, a.C, j, gw, gb);
}

}  // namespace
}  // namespace e2f

using namespace e2f;

extern "C" size_t e2f_layer_norm_backward_workspace_size(int64_t n_atoms, const e2f_norm_cfg* cfg) {
    if (check_norm_cfg(cfg) != E2F_OK || n_atoms < 0) return 0;
    if (n_atoms == 0) return 256;
    if (cfg->C <= kTeamC) return align_up(4 * (size_t)(2 * (kTeamBlocks + kMaxL)) * cfg->C, 256);
    return align_up(4 * (size_t)rows_blocks(n_atoms, cfg->L, cfg->C) * ((cfg->L + 1) * (cfg->L + 1) + 1) * cfg->C, 256);
}

extern "C" e2f_status e2f_layer_norm_backward(const e2f_norm_cfg* cfg, int64_t n_atoms, const void* x,
                                              const uint8_t* x_scales, const float* weight, const float* mean,
                                              const float* rstd, const float* grad_y, const float* grad_skip,
                                              float* grad_x, float* grad_weight, float* grad_bias, void* workspace,
                                              size_t ws_bytes, void* stream_) {
    e2f_status st = check_norm_cfg(cfg);
    if (st != E2F_OK) return st;
    if (n_atoms < 0 || n_atoms > INT32_MAX) return E2F_ERR_INVALID_ARG;
    const bool coded = cfg->x_dtype == E2F_MXI8;
    cudaStream_t s = static_cast<cudaStream_t>(stream_);
    if (misaligned(grad_weight) || misaligned(grad_bias)) return E2F_ERR_ALIGNMENT;
    if (n_atoms == 0) {
        if (grad_weight) E2F_CUDA_TRY(cudaMemsetAsync(grad_weight, 0, 4 * (size_t)(cfg->L + 1) * cfg->C, s));
        if (grad_bias) E2F_CUDA_TRY(cudaMemsetAsync(grad_bias, 0, 4 * (size_t)cfg->C, s));
        return E2F_OK;
    }
    if (!x || !weight || !mean || !rstd || !grad_y || !grad_x || !workspace || (coded && !x_scales))
        return E2F_ERR_INVALID_ARG;
    if (misaligned(x) || misaligned(weight) || misaligned(grad_y) || misaligned(grad_skip) || misaligned(grad_x) ||
        reinterpret_cast<uintptr_t>(workspace) % 256)
        return E2F_ERR_ALIGNMENT;
    if (ws_bytes < e2f_layer_norm_backward_workspace_size(n_atoms, cfg)) return E2F_ERR_INVALID_ARG;
    NormBwdArgs a{n_atoms, cfg->L, cfg->C, ck_blocks(cfg->C), 1.f / cfg->C, x, x_scales, weight, mean, rstd, grad_y, grad_skip,
                  grad_x, grad_weight || grad_bias ? static_cast<float*>(workspace) : nullptr, 0};
    E2F_CUDA_TRY(coded                       ? launch_bwd<kMXI8>(a, grad_weight, grad_bias, s)
                 : cfg->x_dtype == E2F_BF16 ? launch_bwd<kBF16>(a, grad_weight, grad_bias, s)
                                             : launch_bwd<kF32>(a, grad_weight, grad_bias, s));
    return E2F_OK;
}
