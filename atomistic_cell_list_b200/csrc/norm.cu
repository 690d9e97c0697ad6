// Layer norm of irreducible features, forward and backward.
//
// Per node and degree l, over the group of (2l+1) rows of C channels:
//   d = h - mean_c h[0]  (l = 0),  d = h  (l >= 1);   r = 1/sqrt(mean d^2 + eps)
//   y = weight[l,c] d r  (+ bias[c] for l = 0)
// and with xh = d r, u = grad_y weight:
//   grad_x = r (u - xh mean(u xh)  [- mean u for l = 0]) (+ grad_skip)
//   grad_weight[l,c] = sum_{n,m} grad_y xh,   grad_bias[c] = sum_n grad_y[n,0,c]
// All sums are fp32. The work is a few operations per value: memory bound.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "feature_io.cuh"

namespace e2f {
namespace {

constexpr int kMaxNormC = 16384;
constexpr int kNormBlocks = 592;  // most blocks of a weight-gradient pass: 4 on each of 148 SMs

struct NormArgs {
    int64_t n;
    int L, C, nb;
    float eps;
    const void* x;
    const uint8_t* xs;
    const float* res;
    void* sum;
    const float* w;
    const float* b;
    void* y;
    float* mean;
    float* rstd;
    int8_t* codes;
    uint8_t* scales;
};

struct NormBwdArgs {
    int64_t n;
    int L, C, nb;
    const void* x;
    const uint8_t* xs;
    const float* w;
    const float* mean;
    const float* rstd;
    const float* gy;
    const float* skip;
    float* gx;
    float* part;  // weight-gradient partials (null: not wanted)
    int g;        // blocks per row of features: degree l has g (2l+1) blocks
};

// sum over the block, the same value in every thread; sh holds 32 floats and is free again on return
__device__ __forceinline__ float block_sum(float v, float* sh) {
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (nw == 1) return v;
    if (lane == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < nw ? sh[lane] : 0.f;
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    return v;
}

// One block per (node, degree); any C.
template <int XT, int YT, int V>
__global__ void k_norm_rows(NormArgs a) {
    __shared__ float sh[32];
    const int K = (a.L + 1) * (a.L + 1), T = blockDim.x;
    const int iters = (a.C + T * V - 1) / (T * V);
    for (int64_t t = blockIdx.x; t < a.n * (a.L + 1); t += gridDim.x) {
        const int64_t node = t / (a.L + 1);
        const int l = (int)(t % (a.L + 1)), rows = 2 * l + 1;
        const int64_t row0 = node * K + l * l;
        const void* src = a.res ? a.sum : a.x;  // after pass 0 the sum holds what is normalised
        float s = 0.f;
        if (a.res || l == 0 || a.codes) {
            for (int m = 0; m < rows; ++m)
                for (int i = 0; i < iters; ++i) {
                    const int c = (i * T + threadIdx.x) * V;
                    const bool ok = c < a.C;
                    float v[V] = {};
                    if (ok) {
                        load_feat<XT, V>(a.x, a.xs, row0 + m, a.C, a.nb, c, v);
                        if constexpr (XT != kMXI8)
                            if (a.res) {
                                float r[V];
                                load_vec<kF32, V>(a.res, (row0 + m) * a.C + c, r);
                                for (int k = 0; k < V; ++k) v[k] = as_stored<XT>(v[k] + r[k]);
                                store_vec<XT, V>(a.sum, (row0 + m) * a.C + c, v);
                            }
                        for (int k = 0; k < V; ++k) s += v[k];
                    }
                    if constexpr (XT != kMXI8)
                        if (a.codes) store_codes<V>(a.codes, a.scales, row0 + m, a.C, a.nb, c, ok, 32, v);
                }
        }
        const float mu = l == 0 ? block_sum(s, sh) / a.C : 0.f;
        float q = 0.f;
        for (int m = 0; m < rows; ++m)
            for (int c = threadIdx.x * V; c < a.C; c += T * V) {
                float v[V];
                load_feat<XT, V>(src, a.xs, row0 + m, a.C, a.nb, c, v);
                for (int k = 0; k < V; ++k) q += (v[k] - mu) * (v[k] - mu);
            }
        q = block_sum(q, sh);
        const float r = 1.f / sqrtf(q / ((float)rows * a.C) + a.eps);
        for (int m = 0; m < rows; ++m)
            for (int c = threadIdx.x * V; c < a.C; c += T * V) {
                float v[V], w[V], b[V] = {};
                load_feat<XT, V>(src, a.xs, row0 + m, a.C, a.nb, c, v);
                load_vec<kF32, V>(a.w, (int64_t)l * a.C + c, w);
                if (l == 0 && a.b) load_vec<kF32, V>(a.b, c, b);
                for (int k = 0; k < V; ++k) v[k] = (v[k] - mu) * r * w[k] + b[k];
                store_vec<YT, V>(a.y, (row0 + m) * a.C + c, v);
            }
        if (threadIdx.x == 0) {
            if (l == 0 && a.mean) a.mean[node] = mu;
            if (a.rstd) a.rstd[t] = r;
        }
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

// Sums the blocks' partials: rows [g l^2, g (l+1)^2) of part for degree l, [g K, g (K+1)) for the bias.
__global__ void k_norm_join(const float* part, int L, int C, int g, float* gw, float* gb) {
    __shared__ float sh[8][33];
    const int l = blockIdx.y, K = (L + 1) * (L + 1);
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    float* out = l <= L ? gw : gb;
    if (!out) return;
    const int r0 = l <= L ? g * l * l : g * K, r1 = l <= L ? g * (l + 1) * (l + 1) : g * (K + 1);
    float s = 0.f;
    if (c < C)
        for (int r = r0 + w; r < r1; r += 8) s += part[(int64_t)r * C + c];
    sh[w][threadIdx.x & 31] = s;
    __syncthreads();
    if (w == 0 && c < C) {
        for (int k = 1; k < 8; ++k) s += sh[k][threadIdx.x];
        out[(l <= L ? (int64_t)l * C : 0) + c] = s;
    }
}

int row_threads(int C, int V) {
    int t = 32;
    while (t < 512 && t * V < C) t *= 2;
    return t;
}

template <int XT, int YT>
cudaError_t launch_fwd(const NormArgs& a, cudaStream_t s) {
    const int64_t tasks = a.n * (a.L + 1);
    const unsigned grid = (unsigned)std::min<int64_t>(tasks, 1 << 20);
    count_launch();
    if (a.C % 4 == 0)
        k_norm_rows<XT, YT, 4><<<grid, row_threads(a.C, 4), 0, s>>>(a);
    else
        k_norm_rows<XT, YT, 1><<<grid, row_threads(a.C, 1), 0, s>>>(a);
    return cudaGetLastError();
}

template <int XT>
cudaError_t launch_fwd_y(const NormArgs& a, bool y_bf16, cudaStream_t s) {
    return y_bf16 ? launch_fwd<XT, kBF16>(a, s) : launch_fwd<XT, kF32>(a, s);
}

template <int XT, int V>
cudaError_t launch_bwd_v(const NormBwdArgs& a, cudaStream_t s) {
    const size_t smem = a.part ? 8 * (size_t)a.C : 0;
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(k_norm_bwd_rows<XT, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             8 * kMaxNormC);
        if (e != cudaSuccess) return e;
    }
    count_launch();
    k_norm_bwd_rows<XT, V><<<a.g * (a.L + 1) * (a.L + 1), row_threads(a.C, V), smem, s>>>(a);
    return cudaGetLastError();
}

template <int XT>
cudaError_t launch_bwd(const NormBwdArgs& a, cudaStream_t s) {
    return a.C % 4 == 0 ? launch_bwd_v<XT, 4>(a, s) : launch_bwd_v<XT, 1>(a, s);
}

e2f_status check_norm_cfg(const e2f_norm_cfg* c) {
    if (!c) return E2F_ERR_INVALID_ARG;
    if (c->L < 0 || c->C <= 0 || !(c->eps > 0.f) || !std::isfinite(c->eps)) return E2F_ERR_INVALID_ARG;
    if (c->x_dtype != E2F_F32 && c->x_dtype != E2F_BF16 && c->x_dtype != E2F_MXI8) return E2F_ERR_UNSUPPORTED;
    if (c->y_dtype != E2F_F32 && c->y_dtype != E2F_BF16) return E2F_ERR_UNSUPPORTED;
    if (c->L > kMaxL || c->C > kMaxNormC) return E2F_ERR_UNSUPPORTED;
    return E2F_OK;
}

bool misaligned(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 != 0; }

}  // namespace
}  // namespace e2f

using namespace e2f;

extern "C" e2f_status e2f_layer_norm(const e2f_norm_cfg* cfg, int64_t n_atoms, const void* x, const uint8_t* x_scales,
                                     const float* residual, const float* weight, const float* bias, void* sum, void* y,
                                     float* mean, float* rstd, int8_t* ck_codes, uint8_t* ck_scales, void* stream_) {
    e2f_status st = check_norm_cfg(cfg);
    if (st != E2F_OK) return st;
    if (n_atoms < 0 || n_atoms > INT32_MAX) return E2F_ERR_INVALID_ARG;
    const bool coded = cfg->x_dtype == E2F_MXI8;
    if (coded && (residual || ck_codes)) return E2F_ERR_UNSUPPORTED;
    if ((residual != nullptr) != (sum != nullptr) || (ck_codes != nullptr) != (ck_scales != nullptr))
        return E2F_ERR_INVALID_ARG;
    if (n_atoms == 0) return E2F_OK;
    if (!x || !weight || !y || (coded && !x_scales)) return E2F_ERR_INVALID_ARG;
    if (y == x || y == residual || (sum && (y == sum || residual == sum))) return E2F_ERR_INVALID_ARG;
    if (misaligned(x) || misaligned(residual) || misaligned(weight) || misaligned(bias) || misaligned(sum) ||
        misaligned(y) || misaligned(ck_codes))
        return E2F_ERR_ALIGNMENT;
    NormArgs a{n_atoms, cfg->L, cfg->C, ck_blocks(cfg->C), cfg->eps, x,    x_scales, residual,
               sum,     weight, bias,   y,                 mean,     rstd, ck_codes, ck_scales};
    cudaStream_t s = static_cast<cudaStream_t>(stream_);
    const bool yb = cfg->y_dtype == E2F_BF16;
    E2F_CUDA_TRY(coded                       ? launch_fwd_y<kMXI8>(a, yb, s)
                 : cfg->x_dtype == E2F_BF16 ? launch_fwd_y<kBF16>(a, yb, s)
                                             : launch_fwd_y<kF32>(a, yb, s));
    return E2F_OK;
}

extern "C" size_t e2f_layer_norm_backward_workspace_size(int64_t n_atoms, const e2f_norm_cfg* cfg) {
    if (check_norm_cfg(cfg) != E2F_OK || n_atoms < 0) return 0;
    const int K = (cfg->L + 1) * (cfg->L + 1);
    const int64_t g = std::max<int64_t>(1, std::min<int64_t>(n_atoms, kNormBlocks / K));
    return align_up(4 * (size_t)g * (K + 1) * cfg->C, 256);
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
    const int K = (cfg->L + 1) * (cfg->L + 1);
    NormBwdArgs a{n_atoms, cfg->L, cfg->C, ck_blocks(cfg->C), x, x_scales, weight, mean, rstd, grad_y, grad_skip,
                  grad_x,
                  grad_weight || grad_bias ? static_cast<float*>(workspace) : nullptr,
                  (int)std::max<int64_t>(1, std::min<int64_t>(n_atoms, kNormBlocks / K))};
    E2F_CUDA_TRY(coded                       ? launch_bwd<kMXI8>(a, s)
                 : cfg->x_dtype == E2F_BF16 ? launch_bwd<kBF16>(a, s)
                                             : launch_bwd<kF32>(a, s));
    if (a.part) {
        count_launch();
        k_norm_join<<<dim3((cfg->C + 31) / 32, cfg->L + 2), 256, 0, s>>>(a.part, cfg->L, cfg->C, a.g, grad_weight,
                                                                         grad_bias);
        E2F_CUDA_TRY(cudaGetLastError());
    }
    return E2F_OK;
}
