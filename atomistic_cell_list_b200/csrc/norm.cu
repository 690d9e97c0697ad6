// Layer norm of irreducible features: forward (the mathematics and the layout are in norm.cuh).
#include "norm.cuh"

namespace e2f {
namespace {

template <int XT, int YT, int NI, int l>
__device__ __forceinline__ void norm_unit(const NormArgs& a, int64_t node0, int64_t end, int TL) {
    constexpr int R = 2 * l + 1, B = nodes_of(l, fwd_rows(NI)), V = 4;
    const int lane = threadIdx.x & 31, t = lane & (TL - 1), teams = 32 / TL, K = (a.L + 1) * (a.L + 1);
    const int64_t first = node0 + lane / TL;  // a warp's teams take every `teams`-th node
    const int have = (int)min((int64_t)B * teams, end - first);  // node b exists: b teams < have
    // loads are not predicated: a missing node reads the chunk's last one, a lane beyond the row its first
    // channels, so that all of a unit's loads are in flight at once
    bool in[NI];
    int row[B], off[B][NI];
    const int64_t row0 = min(first, end - 1) * K + l * l, base = row0 * a.C;
#pragma unroll
    for (int i = 0; i < NI; ++i) in[i] = (t + TL * i) * V < a.C;
#pragma unroll
    for (int b = 0; b < B; ++b) {
        row[b] = b * teams < have ? b * teams * K : 0;
#pragma unroll
        for (int i = 0; i < NI; ++i) off[b][i] = row[b] * a.C + (in[i] ? (t + TL * i) * V : 0);
    }
    float v[B][R][NI][V];
    {
        Raw4<XT> raw[B][R][NI];
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int m = 0; m < R; ++m)
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    raw[b][m][i].load(a.x, a.xs, base + (off[b][i] + m * a.C),
                                      (row0 + row[b] + m) * a.nb + (in[i] ? (t + TL * i) * V / kCkBlock : 0));
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int m = 0; m < R; ++m)
#pragma unroll
                for (int i = 0; i < NI; ++i) raw[b][m][i].get(v[b][m][i]);
    }
    if constexpr (XT != kMXI8) {
        if (a.res) {
            float4 r[B][R][NI];
#pragma unroll
            for (int b = 0; b < B; ++b)
#pragma unroll
                for (int m = 0; m < R; ++m)
#pragma unroll
                    for (int i = 0; i < NI; ++i)
                        r[b][m][i] = *reinterpret_cast<const float4*>(a.res + base + (off[b][i] + m * a.C));
#pragma unroll
            for (int b = 0; b < B; ++b)
#pragma unroll
                for (int m = 0; m < R; ++m)
#pragma unroll
                    for (int i = 0; i < NI; ++i) {
                        float (&h)[V] = v[b][m][i];
                        h[0] = as_stored<XT>(h[0] + r[b][m][i].x);
                        h[1] = as_stored<XT>(h[1] + r[b][m][i].y);
                        h[2] = as_stored<XT>(h[2] + r[b][m][i].z);
                        h[3] = as_stored<XT>(h[3] + r[b][m][i].w);
                        if (b * teams < have && in[i]) store_vec<XT, V>(a.sum, base + (off[b][i] + m * a.C), h);
                    }
        }
        if (a.codes)
#pragma unroll
            for (int b = 0; b < B; ++b)
#pragma unroll
                for (int m = 0; m < R; ++m)
#pragma unroll
                    for (int i = 0; i < NI; ++i)
                        store_codes<V>(a.codes, a.scales, row0 + row[b] + m, a.C, a.nb, (t + TL * i) * V,
                                       b * teams < have && in[i], TL, v[b][m][i]);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i)
        if (!in[i])
#pragma unroll
            for (int b = 0; b < B; ++b)
#pragma unroll
                for (int m = 0; m < R; ++m)
                    for (int k = 0; k < V; ++k) v[b][m][i][k] = 0.f;
    float mu[B], q[B];
    if constexpr (l == 0) {
#pragma unroll
        for (int b = 0; b < B; ++b) {
            mu[b] = 0.f;
#pragma unroll
            for (int i = 0; i < NI; ++i)
                for (int k = 0; k < V; ++k) mu[b] += v[b][0][i][k];
        }
        team_sum(mu, TL);
#pragma unroll
        for (int b = 0; b < B; ++b) {
            mu[b] /= a.C;
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (in[i])
                    for (int k = 0; k < V; ++k) v[b][0][i][k] -= mu[b];
        }
    }
#pragma unroll
    for (int b = 0; b < B; ++b) {
        q[b] = 0.f;
#pragma unroll
        for (int m = 0; m < R; ++m)
#pragma unroll
            for (int i = 0; i < NI; ++i)
                for (int k = 0; k < V; ++k) q[b] += v[b][m][i][k] * v[b][m][i][k];
    }
    team_sum(q, TL);
#pragma unroll
    for (int b = 0; b < B; ++b) q[b] = 1.f / sqrtf(q[b] / ((float)R * a.C) + a.eps);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        if (!in[i]) continue;
        const int c = (t + TL * i) * V;
        float w[V], bias[V] = {};
        load_vec<kF32, V>(a.w, l * a.C + c, w);
        if (l == 0 && a.b) load_vec<kF32, V>(a.b, c, bias);
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int m = 0; m < R; ++m)
                if (b * teams < have) {
                    float y[V];
                    for (int k = 0; k < V; ++k) y[k] = v[b][m][i][k] * q[b] * w[k] + bias[k];
                    store_vec<YT, V>(a.y, base + (off[b][i] + m * a.C), y);
                }
    }
    if (t == 0)
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (b * teams < have) {
                const int64_t node = first + b * teams;
                if (l == 0 && a.mean) a.mean[node] = mu[b];
                if (a.rstd) a.rstd[node * (a.L + 1) + l] = q[b];
            }
}

template <int XT, int YT, int NI>
__global__ void __launch_bounds__(256, NI == 1 ? 2 : 1) k_norm_teams(NormArgs a, int TL, int S, Units un) {
    const int teams = 32 / TL;
    const int64_t c0 = (int64_t)blockIdx.x * S, end = min(c0 + S, a.n);
    for (int u = threadIdx.x >> 5; u < un.total; u += 8) {
        int j = u, l = kMaxL;  // the largest degrees first
        while (j >= un.n[l]) j -= un.n[l--];
        j *= teams;
        switch (l) {
            case 0: norm_unit<XT, YT, NI, 0>(a, c0 + j * nodes_of(0, fwd_rows(NI)), end, TL); break;
            case 1: norm_unit<XT, YT, NI, 1>(a, c0 + j * nodes_of(1, fwd_rows(NI)), end, TL); break;
            case 2: norm_unit<XT, YT, NI, 2>(a, c0 + j * nodes_of(2, fwd_rows(NI)), end, TL); break;
            case 3: norm_unit<XT, YT, NI, 3>(a, c0 + j * nodes_of(3, fwd_rows(NI)), end, TL); break;
            default: norm_unit<XT, YT, NI, 4>(a, c0 + j * nodes_of(4, fwd_rows(NI)), end, TL); break;
        }
    }
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

template <int XT, int YT>
cudaError_t launch_fwd(const NormArgs& a, cudaStream_t s) {
    count_launch();
    if (use_teams(a.C)) {
        const TeamPlan p = team_plan(a.n, a.L, a.C, 4 * kSMs, true);
        if (p.NI == 1) k_norm_teams<XT, YT, 1><<<(unsigned)p.chunks, 256, 0, s>>>(a, p.TL, p.S, p.un);
        else k_norm_teams<XT, YT, 2><<<(unsigned)p.chunks, 256, 0, s>>>(a, p.TL, p.S, p.un);
        return cudaGetLastError();
    }
    const unsigned grid = (unsigned)std::min<int64_t>(a.n * (a.L + 1), 1 << 20);
    if (a.C % 4 == 0) k_norm_rows<XT, YT, 4><<<grid, row_threads(a.C, 4), 0, s>>>(a);
    else k_norm_rows<XT, YT, 1><<<grid, row_threads(a.C, 1), 0, s>>>(a);
    return cudaGetLastError();
}

template <int XT>
cudaError_t launch_fwd_y(const NormArgs& a, bool y_bf16, cudaStream_t s) {
    return y_bf16 ? launch_fwd<XT, kBF16>(a, s) : launch_fwd<XT, kF32>(a, s);
}

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
