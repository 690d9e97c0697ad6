// Layer norm of irreducible features: backward (the mathematics and the layout are in norm.cuh).
#include "norm.cuh"

namespace e2f {
namespace {

constexpr int kBwdBlocks = 2 * kSMs;  // resident blocks of k_norm_bwd_teams

// acc: this lane's weight gradient of its channels, [degree or bias][NI] float4 with a stride of 32 float4
template <int XT, int NI, int l>
__device__ __forceinline__ void norm_bwd_unit(const NormBwdArgs& a, int64_t node0, int64_t end, int TL, float4* acc) {
    constexpr int R = 2 * l + 1, B = nodes_of(l, bwd_rows(NI)), V = 4;
    const int lane = threadIdx.x & 31, t = lane & (TL - 1), teams = 32 / TL, K = (a.L + 1) * (a.L + 1);
    const int64_t first = node0 + lane / TL;
    const int have = (int)min((int64_t)B * teams, end - first);
    bool in[NI];  // unpredicated loads, as in the forward
    int row[B], off[B][NI];
    const int64_t node_at = min(first, end - 1), row0 = node_at * K + l * l, base = row0 * a.C;
#pragma unroll
    for (int i = 0; i < NI; ++i) in[i] = (t + TL * i) * V < a.C;
#pragma unroll
    for (int b = 0; b < B; ++b) {
        row[b] = b * teams < have ? b * teams * K : 0;
#pragma unroll
        for (int i = 0; i < NI; ++i) off[b][i] = row[b] * a.C + (in[i] ? (t + TL * i) * V : 0);
    }
    float x[B][R][NI][V], g[B][R][NI][V], mu[B], r[B], s1[B], s2[B];
    {
        Raw4<XT> raw[B][R][NI];
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int m = 0; m < R; ++m)
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    raw[b][m][i].load(a.x, a.xs, base + (off[b][i] + m * a.C),
                                      (row0 + row[b] + m) * a.nb + (in[i] ? (t + TL * i) * V / kCkBlock : 0));
                    load_vec<kF32, V>(a.gy, base + (off[b][i] + m * a.C), g[b][m][i]);
                }
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int64_t node = node_at + (b * teams < have ? b * teams : 0);
            mu[b] = l == 0 ? a.mean[node] : 0.f;
            r[b] = a.rstd[node * (a.L + 1) + l];
            s1[b] = s2[b] = 0.f;
        }
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int m = 0; m < R; ++m)
#pragma unroll
                for (int i = 0; i < NI; ++i) raw[b][m][i].get(x[b][m][i]);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        if (!in[i]) continue;
        float w[V], dw[V] = {}, db[V] = {};
        load_vec<kF32, V>(a.w, l * a.C + (t + TL * i) * V, w);
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (b * teams < have)
#pragma unroll
                for (int m = 0; m < R; ++m)
                    for (int k = 0; k < V; ++k) {
                        const float gk = g[b][m][i][k], u = gk * w[k];
                        const float xh = (l == 0 ? x[b][m][i][k] - mu[b] : x[b][m][i][k]) * r[b];
                        dw[k] += gk * xh;
                        s2[b] += u * xh;
                        if constexpr (l == 0) {
                            db[k] += gk;
                            s1[b] += u;
                        }
                        x[b][m][i][k] = xh;
                        g[b][m][i][k] = u;
                    }
        if (a.part) {
            float4& o = acc[(l * NI + i) * 32];
            o = make_float4(o.x + dw[0], o.y + dw[1], o.z + dw[2], o.w + dw[3]);
            if constexpr (l == 0) {
                float4& p = acc[((a.L + 1) * NI + i) * 32];
                p = make_float4(p.x + db[0], p.y + db[1], p.z + db[2], p.w + db[3]);
            }
        }
    }
    if constexpr (l == 0) team_sum(s1, TL);
    team_sum(s2, TL);
#pragma unroll
    for (int b = 0; b < B; ++b) {
        s1[b] /= a.C;
        s2[b] /= (float)R * a.C;
#pragma unroll
        for (int m = 0; m < R; ++m)
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (b * teams < have && in[i]) {
                    const int64_t at = base + (off[b][i] + m * a.C);
                    float d[V];
                    for (int k = 0; k < V; ++k)
                        d[k] = r[b] * (g[b][m][i][k] - (l == 0 ? s1[b] : 0.f) - x[b][m][i][k] * s2[b]);
                    if (a.skip) {
                        float e[V];
                        load_vec<kF32, V>(a.skip, at, e);
                        for (int k = 0; k < V; ++k) d[k] += e[k];
                    }
                    store_vec<kF32, V>(a.gx, at, d);
                }
    }
}

// Persistent blocks: block b takes chunks b, b + grid, ..., its warps the units
// of those chunks in turn. The weight gradient stays in shared memory, one
// private slot per lane, degree and channel, until the block's end: no atomics,
// one fixed order.
template <int XT, int NI>
__global__ void __launch_bounds__(256, NI == 1 ? 2 : 1) k_norm_bwd_teams(NormBwdArgs a, int TL, int S, Units un,
                                                                         int64_t chunks) {
    extern __shared__ float4 acc4[];  // [8 warps][L + 2][NI][32 lanes]
    const int teams = 32 / TL, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per_warp = (a.L + 2) * NI * 32;
    float4* acc = acc4 + warp * per_warp + lane;
    for (int k = 0; k < (a.L + 2) * NI; ++k) acc[k * 32] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int64_t mine = (chunks - blockIdx.x + gridDim.x - 1) / gridDim.x * un.total;  // units of this block
    for (int64_t k = warp; k < mine; k += 8) {
        const int64_t c0 = (blockIdx.x + k / un.total * gridDim.x) * S, end = min(c0 + S, a.n);
        int j = (int)(k % un.total), l = kMaxL;
        while (j >= un.n[l]) j -= un.n[l--];
        j *= teams;
        switch (l) {
            case 0: norm_bwd_unit<XT, NI, 0>(a, c0 + j * nodes_of(0, bwd_rows(NI)), end, TL, acc); break;
            case 1: norm_bwd_unit<XT, NI, 1>(a, c0 + j * nodes_of(1, bwd_rows(NI)), end, TL, acc); break;
            case 2: norm_bwd_unit<XT, NI, 2>(a, c0 + j * nodes_of(2, bwd_rows(NI)), end, TL, acc); break;
            case 3: norm_bwd_unit<XT, NI, 3>(a, c0 + j * nodes_of(3, bwd_rows(NI)), end, TL, acc); break;
            default: norm_bwd_unit<XT, NI, 4>(a, c0 + j * nodes_of(4, bwd_rows(NI)), end, TL, acc); break;
        }
    }
    if (!a.part) return;
    __syncthreads();
    // the block's sums over its warps and their teams, in order
    const float* f = reinterpret_cast<const float*>(acc4);
    for (int o = threadIdx.x; o < (a.L + 2) * a.C; o += 256) {
        const int l = o / a.C, c = o % a.C, v = c / 4, i = v / TL, t = v % TL;
        float s = 0.f;
        for (int w = 0; w < 8; ++w)
            for (int q = 0; q < teams; ++q) s += f[(w * per_warp + (l * NI + i) * 32 + q * TL + t) * 4 + c % 4];
        a.part[(int64_t)blockIdx.x * (a.L + 2) * a.C + o] = s;
    }
}

// One block per (node, degree), the blocks split over the degrees as the rows
// are: degree l has blocks [g l^2, g (l+1)^2). Each thread owns its channels,
// so the block's part of the weight gradient is summed in shared memory
// without atomics, in a fixed order.
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

// Sums the blocks' partials: `count` rows of `stride` values for each degree and the bias.
struct JoinPlan {
    int64_t base[kMaxL + 2], stride;
    int count[kMaxL + 2];
};

__global__ void __launch_bounds__(1024) k_norm_join(const float* part, int L, int C, JoinPlan p, float* gw, float* gb) {
    __shared__ float sh[32][33];
    const int l = blockIdx.y, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane, w = threadIdx.x >> 5;
    float* out = l <= L ? gw : gb;
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
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(k_norm_bwd_rows<XT, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             8 * kMaxNormC);
        if (e != cudaSuccess) return e;
    }
    k_norm_bwd_rows<XT, V><<<a.g * (a.L + 1) * (a.L + 1), row_threads(a.C, V), smem, s>>>(a);
    return cudaGetLastError();
}

template <int XT, int NI>
cudaError_t launch_bwd_teams(const NormBwdArgs& a, const TeamPlan& p, int blocks, cudaStream_t s) {
    const size_t smem = 8 * (size_t)(a.L + 2) * NI * 32 * sizeof(float4);
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(k_norm_bwd_teams<XT, NI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)smem);
        if (e != cudaSuccess) return e;
    }
    k_norm_bwd_teams<XT, NI><<<blocks, 256, smem, s>>>(a, p.TL, p.S, p.un, p.chunks);
    return cudaGetLastError();
}

// blocks of a backward call: rows of partials (teams), or blocks per row of features
int bwd_blocks(int64_t n, int L, int C) {
    if (use_teams(C)) return (int)std::min<int64_t>(team_plan(n, L, C, kBwdBlocks, false).chunks, kBwdBlocks);
    return (int)std::max<int64_t>(1, std::min<int64_t>(n, kNormBlocks / ((L + 1) * (L + 1))));
}

template <int XT>
cudaError_t launch_bwd(NormBwdArgs a, float* gw, float* gb, cudaStream_t s) {
    const int K = (a.L + 1) * (a.L + 1), blocks = bwd_blocks(a.n, a.L, a.C);
    JoinPlan j{};
    cudaError_t e;
    count_launch();
    if (use_teams(a.C)) {
        const TeamPlan p = team_plan(a.n, a.L, a.C, kBwdBlocks, false);
        e = p.NI == 1 ? launch_bwd_teams<XT, 1>(a, p, blocks, s) : launch_bwd_teams<XT, 2>(a, p, blocks, s);
        j.stride = (int64_t)(a.L + 2) * a.C;
        for (int l = 0; l < a.L + 2; ++l) {
            j.base[l] = (int64_t)l * a.C;
            j.count[l] = blocks;
        }
    } else {
        a.g = blocks;
        e = a.C % 4 == 0 ? launch_bwd_rows<XT, 4>(a, s) : launch_bwd_rows<XT, 1>(a, s);
        j.stride = a.C;
        for (int l = 0; l < a.L + 2; ++l) {
            j.base[l] = (int64_t)a.g * (l <= a.L ? l * l : K) * a.C;
            j.count[l] = a.g * (l <= a.L ? 2 * l + 1 : 1);
        }
    }
    if (e != cudaSuccess || !a.part) return e;
    count_launch();
    k_norm_join<<<dim3((a.C + 31) / 32, a.L + 2), 1024, 0, s>>>(a.part, a.L, a.C, j, gw, gb);
    return cudaGetLastError();
}

}  // namespace
}  // namespace e2f

using namespace e2f;

extern "C" size_t e2f_layer_norm_backward_workspace_size(int64_t n_atoms, const e2f_norm_cfg* cfg) {
    if (check_norm_cfg(cfg) != E2F_OK || n_atoms < 0) return 0;
    if (n_atoms == 0) return 256;
    const int rows = use_teams(cfg->C) ? cfg->L + 2 : (cfg->L + 1) * (cfg->L + 1) + 1;
    return align_up(4 * (size_t)bwd_blocks(n_atoms, cfg->L, cfg->C) * rows * cfg->C, 256);
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
    NormBwdArgs a{n_atoms, cfg->L, cfg->C, ck_blocks(cfg->C), x, x_scales, weight, mean, rstd, grad_y, grad_skip,
                  grad_x, grad_weight || grad_bias ? static_cast<float*>(workspace) : nullptr, 0};
    E2F_CUDA_TRY(coded                       ? launch_bwd<kMXI8>(a, grad_weight, grad_bias, s)
                 : cfg->x_dtype == E2F_BF16 ? launch_bwd<kBF16>(a, grad_weight, grad_bias, s)
                                             : launch_bwd<kF32>(a, grad_weight, grad_bias, s));
    return E2F_OK;
}
