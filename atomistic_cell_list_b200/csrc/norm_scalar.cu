// Layer norm of irreducible features for up to 256 channels that are no multiple of 4: rows begin on any 4 (fp32),
// 2 (bf16) or 1 (codes) bytes, so values are loaded one by one. One warp per unit of up to 9 rows, a lane owns the
// channels lane + 32 i, i < NI, and holds them for all rows of the unit; blocks work on one degree (norm.cuh). All
// loads of a unit are in flight together. fp32 moves 128 bytes an instruction; instructions bound it, and spills where
// a lane holds more than its registers: bf16 forward 290 bytes up to 128 channels, 1,600 above; backward above 128
// channels 220 (fp32) to 1,700 (codes). A skip gradient, which grad_x may overwrite, is loaded value by value between
// the stores. 20,000 atoms, L = 4, C = 101, fp32: forward 93 us, backward 218 us, with a skip gradient 803 us (C = 100
// with its 16-byte pieces: 82, 119 and 153 us); from bf16 to bf16 105 us; from codes 143 us, their backward with a
// skip gradient 884 us. 8,000 atoms, C = 255: forward from bf16 155 us, backward of fp32 216 us, with a skip 836 us.
#include "norm.cuh"

namespace e2f {
namespace {

constexpr int kWarps = 4;  // of a block

__host__ __device__ constexpr int scalar_nodes(int l, int NI) { return NI <= 4 ? unit_nodes(l) : l == 0 ? 4 : 1; }

// one value: row r of a unit that begins at row0 (base = row0 C), channel c
template <int XT>
__device__ __forceinline__ float value(const void* x, int64_t base, const uint8_t* unit_scales, int r,
                                       int C, int nb, int c) {
    float e[1];
    if constexpr (XT == kMXI8) e[0] = static_cast<const int8_t*>(x)[base + (r * C + c)] *
                                      (ck_scale(unit_scales[r * nb + c / kCkBlock]) * 0.015625f);
    else load_vec<XT, 1>(x, base + (r * C + c), e);
    return e[0];
}

// blocks [at[l], at[l+1]) work on degree l
struct Blocks {
    int at[kMaxL + 2];
};

Blocks blocks_of(int64_t n, int L, int NI, int most) {
    Blocks p{};
    const double rows = (L + 1) * (L + 1) + 0.5 * (L + 1);
    for (int l = 0; l <= L; ++l) {
        const int64_t units = (n + scalar_nodes(l, NI) - 1) / scalar_nodes(l, NI);
        const int share = std::max(1, (int)(most * (2 * l + 1.5) / rows));
        p.at[l + 1] = p.at[l] + (int)std::min<int64_t>(share, units);
    }
    for (int l = L + 1; l <= kMaxL; ++l) p.at[l + 1] = p.at[l];
    return p;
}

template <int XT, int YT, int NI, int l>
__device__ __forceinline__ void scalar_degree(const NormArgs& a, const Blocks& p) {
    constexpr int R = 2 * l + 1, B = scalar_nodes(l, NI);
    const int lane = threadIdx.x & 31, C = a.C, K = (a.L + 1) * (a.L + 1), blocks = p.at[l + 1] - p.at[l];
    int c[NI];
    bool in[NI];
    float w[NI], bias[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        in[i] = lane + 32 * i < C;
        c[i] = in[i] ? lane + 32 * i : 0;
        w[i] = a.w[l * C + c[i]];
        bias[i] = l == 0 && a.b ? a.b[c[i]] : 0.f;
    }
    const int64_t units = (a.n + B - 1) / B;
    for (int64_t k = (int)blockIdx.x - p.at[l] + (int64_t)blocks * (threadIdx.x >> 5); k < units;
         k += (int64_t)blocks * kWarps) {
        const int have = (int)min((int64_t)B, a.n - k * B);
        const int64_t row0 = k * B * K + l * l, base = row0 * C;
        const uint8_t* xs = XT == kMXI8 ? a.xs + row0 * a.nb : nullptr;
        float v[B][R][NI], mu[B], q[B];
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
            for (int m = 0; m < R; ++m)
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const float e = value<XT>(a.x, base, xs, (b < have ? b : 0) * K + m, C, a.nb, c[i]);
                    v[b][m][i] = in[i] ? e : 0.f;
                }
        if constexpr (XT != kMXI8) {
            if (a.res)
#pragma unroll
                for (int b = 0; b < B; ++b)
#pragma unroll
                    for (int m = 0; m < R; ++m)
#pragma unroll
                        for (int i = 0; i < NI; ++i) {
                            const int at = ((b < have ? b : 0) * K + m) * C + c[i];
                            const float h[1] = {as_stored<XT>(v[b][m][i] + a.res[base + at])};
                            if (in[i]) v[b][m][i] = h[0];
                            if (b < have && in[i]) store_vec<XT, 1>(a.sum, base + at, h);
                        }
            if (a.codes)
#pragma unroll
                for (int b = 0; b < B; ++b)
#pragma unroll
                    for (int m = 0; m < R; ++m)
#pragma unroll
                        for (int i = 0; i < NI; ++i) {
                            const float h[1] = {v[b][m][i]};
                            store_codes<1>(a.codes, a.scales, row0 + (b * K + m), C, a.nb, lane + 32 * i,
                                           b < have && in[i], 32, h);
                        }
        }
        if constexpr (l == 0) {
#pragma unroll
            for (int b = 0; b < B; ++b) {
                mu[b] = 0.f;
#pragma unroll
                for (int i = 0; i < NI; ++i) mu[b] += v[b][0][i];
            }
            team_sum(mu, 32);
#pragma unroll
            for (int b = 0; b < B; ++b) {
                mu[b] *= a.inv_c;
#pragma unroll
                for (int i = 0; i < NI; ++i) v[b][0][i] -= in[i] ? mu[b] : 0.f;
            }
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
            q[b] = 0.f;
#pragma unroll
            for (int m = 0; m < R; ++m)
#pragma unroll
                for (int i = 0; i < NI; ++i) q[b] += v[b][m][i] * v[b][m][i];
        }
        team_sum(q, 32);
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (b >= have) continue;
            const float r = rsqrtf(q[b] * (a.inv_c * (1.f / R)) + a.eps);
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (in[i])
#pragma unroll
                    for (int m = 0; m < R; ++m) {
                        const float y[1] = {fmaf(v[b][m][i] * r, w[i], bias[i])};
                        store_vec<YT, 1>(a.y, base + ((b * K + m) * C + c[i]), y);
                    }
            if (lane == 0) {
                const int64_t node = k * B + b;
                if (l == 0 && a.mean) a.mean[node] = mu[b];
                if (a.rstd) a.rstd[node * (a.L + 1) + l] = r;
            }
        }
    }
}

template <int XT, int YT, int NI>
__global__ void __launch_bounds__(32 * kWarps, NI <= 4 ? 3 : 2) k_norm_scalar(NormArgs a, Blocks p) {
    const int blk = blockIdx.x;
    if (blk < p.at[1]) scalar_degree<XT, YT, NI, 0>(a, p);
    else if (blk < p.at[2]) scalar_degree<XT, YT, NI, 1>(a, p);
    else if (blk < p.at[3]) scalar_degree<XT, YT, NI, 2>(a, p);
    else if (blk < p.at[4]) scalar_degree<XT, YT, NI, 3>(a, p);
    else scalar_degree<XT, YT, NI, 4>(a, p);
}

// part: [block][C], then [block of degree 0][C] for the bias
template <int XT, int NI, int l>
__device__ __forceinline__ void scalar_bwd_degree(const NormBwdArgs& a, const Blocks& p) {
    constexpr int R = 2 * l + 1, B = scalar_nodes(l, NI) < 4 ? scalar_nodes(l, NI) : 4;
    __shared__ float sh[kWarps][32 * NI];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, C = a.C, K = (a.L + 1) * (a.L + 1);
    const int blocks = p.at[l + 1] - p.at[l];
    int c[NI];
    bool in[NI];
    float w[NI], dw[NI] = {}, db[NI] = {};
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        in[i] = lane + 32 * i < C;
        c[i] = in[i] ? lane + 32 * i : 0;
        w[i] = a.w[l * C + c[i]];
    }
    const int64_t units = (a.n + B - 1) / B;
    for (int64_t k = (int)blockIdx.x - p.at[l] + (int64_t)blocks * warp; k < units; k += (int64_t)blocks * kWarps) {
        const int have = (int)min((int64_t)B, a.n - k * B);
        const int64_t row0 = k * B * K + l * l, base = row0 * C;
        const uint8_t* xs = XT == kMXI8 ? a.xs + row0 * a.nb : nullptr;
        float x[B][R][NI], g[B][R][NI], r[B], s1[B], s2[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int bb = b < have ? b : 0;
#pragma unroll
            for (int m = 0; m < R; ++m)
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    x[b][m][i] = value<XT>(a.x, base, xs, bb * K + m, C, a.nb, c[i]);
                    g[b][m][i] = a.gy[base + ((bb * K + m) * C + c[i])];
                }
            r[b] = a.rstd[(k * B + bb) * (a.L + 1) + l];
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
            s1[b] = s2[b] = 0.f;
            const float mu = l == 0 ? a.mean[k * B + (b < have ? b : 0)] : 0.f;
#pragma unroll
            for (int m = 0; m < R; ++m)
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    if (in[i]) {
                        const float xh = (l == 0 ? x[b][m][i] - mu : x[b][m][i]) * r[b], gk = g[b][m][i], u = gk * w[i];
                        if (b < have) dw[i] += gk * xh;
                        if (l == 0 && b < have) db[i] += gk;
                        s1[b] += u;
                        s2[b] += u * xh;
                        x[b][m][i] = xh;
                        g[b][m][i] = u;
                    }
        }
        if constexpr (l == 0) team_sum(s1, 32);
        team_sum(s2, 32);
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (b >= have) continue;
            const float m1 = l == 0 ? s1[b] * a.inv_c : 0.f, m2 = s2[b] * (a.inv_c * (1.f / R));
#pragma unroll
            for (int m = 0; m < R; ++m)
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    if (in[i]) {
                        const int64_t at = base + ((b * K + m) * C + c[i]);
                        const float e = a.skip ? a.skip[at] : 0.f;
                        a.gx[at] = e + r[b] * (g[b][m][i] - m1 - x[b][m][i] * m2);
                    }
        }
    }
    if (!a.part) return;
#pragma unroll
    for (int pass = 0; pass < (l == 0 ? 2 : 1); ++pass) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NI; ++i) sh[warp][lane + 32 * i] = pass == 0 ? dw[i] : db[i];
        __syncthreads();
        float* out = a.part + (int64_t)(blockIdx.x + (pass == 0 ? 0 : p.at[kMaxL + 1])) * C;
        for (int o = threadIdx.x; o < C; o += 32 * kWarps) {
            float s = 0.f;
            for (int q = 0; q < kWarps; ++q) s += sh[q][o];
            out[o] = s;
        }
    }
}

template <int XT, int NI>
__global__ void __launch_bounds__(32 * kWarps, 2) k_norm_bwd_scalar(NormBwdArgs a, Blocks p) {
    const int blk = blockIdx.x;
    if (blk < p.at[1]) scalar_bwd_degree<XT, NI, 0>(a, p);
    else if (blk < p.at[2]) scalar_bwd_degree<XT, NI, 1>(a, p);
    else if (blk < p.at[3]) scalar_bwd_degree<XT, NI, 2>(a, p);
    else if (blk < p.at[4]) scalar_bwd_degree<XT, NI, 3>(a, p);
    else scalar_bwd_degree<XT, NI, 4>(a, p);
}

template <int XT, int YT>
cudaError_t fwd(const NormArgs& a, cudaStream_t s) {
    const Blocks p = blocks_of(a.n, a.L, a.C <= 128 ? 4 : 8, (a.C <= 128 ? 3 : 2) * kSMs);
    if (a.C <= 128) k_norm_scalar<XT, YT, 4><<<p.at[kMaxL + 1], 32 * kWarps, 0, s>>>(a, p);
    else k_norm_scalar<XT, YT, 8><<<p.at[kMaxL + 1], 32 * kWarps, 0, s>>>(a, p);
    return cudaGetLastError();
}

template <int XT>
cudaError_t bwd(const NormBwdArgs& a, const Blocks& p, cudaStream_t s) {
    if (a.C <= 128) k_norm_bwd_scalar<XT, 4><<<p.at[kMaxL + 1], 32 * kWarps, 0, s>>>(a, p);
    else k_norm_bwd_scalar<XT, 8><<<p.at[kMaxL + 1], 32 * kWarps, 0, s>>>(a, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t run_norm_scalar(const NormArgs& a, int x_type, bool y_bf16, cudaStream_t s) {
    if (x_type == kF32) return y_bf16 ? fwd<kF32, kBF16>(a, s) : fwd<kF32, kF32>(a, s);
    if (x_type == kBF16) return y_bf16 ? fwd<kBF16, kBF16>(a, s) : fwd<kBF16, kF32>(a, s);
    return y_bf16 ? fwd<kMXI8, kBF16>(a, s) : fwd<kMXI8, kF32>(a, s);
}

cudaError_t run_norm_bwd_scalar(const NormBwdArgs& a, int x_type, int* at, cudaStream_t s) {
    const Blocks p = blocks_of(a.n, a.L, a.C <= 128 ? 4 : 8, kTeamBlocks);
    std::copy(p.at, p.at + kMaxL + 2, at);
    return x_type == kF32 ? bwd<kF32>(a, p, s) : x_type == kBF16 ? bwd<kBF16>(a, p, s) : bwd<kMXI8>(a, p, s);
}

}  // namespace e2f
