// Layer norm of irreducible features: forward (the mathematics and the layout are in norm.cuh).
#include "norm.cuh"

namespace e2f {
namespace {

constexpr int kFwdWarps = 8;  // of a block, at 128 registers

// The units of degree l that this block takes. 3,000 atoms, L = 4, C = 128, fp32
// stream + fp32 residual -> stream and bf16 features: 134 MB in 24 us (5.6 TB/s).
// 20,000 atoms with the checkpoint beside them: 0.96 GB in 170 us. From codes to bf16
// (194 MB in 68 us) it is bound by instructions, 79 per row of 128 values. C above 128
// holds two vectors a lane and spills up to 204 bytes at 128 registers: 12,000 atoms of
// 256 channels, fp32 with a residual, 1.08 GB in 256 us, bf16 307 MB in 99 us, from codes
// 233 MB in 106 us (65, 48 and 34 % of the copy rate).
template <int XT, int YT, int NI, int l>
__device__ __forceinline__ void norm_degree(const NormArgs& a, int TL, const Slots& sl, char* smem) {
    using U = Unit<NI, l>;
    constexpr int V = 4, E = vec_bytes<XT>() / 4, R = U::R, B = U::B;  // E: bytes of a value
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, lane = threadIdx.x & 31, t = lane & (TL - 1), C = a.C;
    const int K = (a.L + 1) * (a.L + 1), teams = 32 / TL, team0 = lane / TL * (B * R);
    const uint32_t smem_s = (uint32_t)__cvta_generic_to_shared(smem);
    const uint32_t zeros = smem_s + warps * sl.stages * sl.stage_bytes;  // what lanes beyond the row read
    const uint32_t mine_s = smem_s + warp * sl.stages * sl.stage_bytes;
    int c[NI];
    bool in[NI];
    float w[NI][V], bias[NI][V] = {};
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        in[i] = (t + TL * i) * V < C;
        c[i] = in[i] ? (t + TL * i) * V : 0;
        load_vec<kF32, V>(a.w, l * C + c[i], w[i]);
        if (l == 0 && a.b) load_vec<kF32, V>(a.b, c[i], bias[i]);
    }
    const int blocks = sl.at[l + 1] - sl.at[l];
    const int64_t step = (int64_t)blocks * warps, units = (a.n + B * teams - 1) / (B * teams);
    int64_t k = (int)blockIdx.x - sl.at[l] + (int64_t)blocks * warp;
    auto fetch = [&](int64_t k, int stage) {
        if (k < units) {
            const U u(k, a.n, K, TL);
            const uint32_t to = mine_s + stage * sl.stage_bytes;
            u.template fetch<XT>(a.x, C, K, TL, to);
            if (XT != kMXI8 && a.res) u.template fetch<kF32>(a.res, C, K, TL, to + sl.o1);
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
        // addresses run along with the rows: a node's rows follow one another, the team's nodes lie jump rows apart
        const int64_t base = u.row0 * C;
        const int jump = teams * K;
        float v[B][R][NI][V];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const uint32_t p = in[i] ? st + (team0 * C + c[i]) * E : zeros;
            const int pitch = in[i] ? C * E : 0;
#pragma unroll
            for (int b = 0; b < B; ++b)
#pragma unroll
                for (int m = 0; m < R; ++m) {
                    Raw4<XT> raw;
                    raw.from(p + (b * R + m) * pitch);
                    if constexpr (XT == kMXI8) raw.s = scale[b * R + m][i];
                    raw.get(v[b][m][i]);
                }
            if constexpr (XT != kMXI8) {
                if (a.res) {
                    const uint32_t r = in[i] ? st + sl.o1 + (team0 * C + c[i]) * 4 : zeros;
                    const int r_pitch = in[i] ? C * 4 : 0;
                    char* sum = static_cast<char*>(a.sum) + (base + c[i]) * E;
#pragma unroll
                    for (int b = 0; b < B; ++b) {
                        char* to = sum;
#pragma unroll
                        for (int m = 0; m < R; ++m) {
                            Raw4<kF32> e;
                            e.from(r + (b * R + m) * r_pitch);
                            float (&h)[V] = v[b][m][i];
                            h[0] = as_stored<XT>(h[0] + e.a.x); h[1] = as_stored<XT>(h[1] + e.a.y);
                            h[2] = as_stored<XT>(h[2] + e.a.z); h[3] = as_stored<XT>(h[3] + e.a.w);
                            if (b < u.have && in[i]) store_vec<XT, V>(to, 0, h);
                            to += C * E;
                        }
                        sum += (int64_t)jump * C * E;
                    }
                }
                if (a.codes) {
                    int8_t* codes = a.codes + base + c[i];
                    uint8_t* scales = a.scales + u.row0 * a.nb + c[i] / kCkBlock;
#pragma unroll
                    for (int b = 0; b < B; ++b) {
                        int8_t* to = codes;
                        uint8_t* to_s = scales;
#pragma unroll
                        for (int m = 0; m < R; ++m) {
                            store_codes_at<V>(to, to_s, c[i] % kCkBlock == 0, b < u.have && in[i], TL, v[b][m][i]);
                            to += C;
                            to_s += a.nb;
                        }
                        codes += (int64_t)jump * C;
                        scales += (int64_t)jump * a.nb;
                    }
                }
            }
        }
        if constexpr (XT == kMXI8)
            if (k + step < units) U(k + step, a.n, K, TL).scales(a.xs, a.nb, K, TL, c, scale);
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
                mu[b] *= a.inv_c;
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    for (int k = 0; k < V; ++k) v[b][0][i][k] -= in[i] ? mu[b] : 0.f;
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
        for (int b = 0; b < B; ++b) {
            q[b] = rsqrtf(q[b] * (a.inv_c * (1.f / R)) + a.eps);
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                float f[V];
                for (int k = 0; k < V; ++k) f[k] = q[b] * w[i][k];
                constexpr int EY = vec_bytes<YT>() / 4;
                char* to = static_cast<char*>(a.y) + (base + (int64_t)(b * jump) * C + c[i]) * EY;
                if (b < u.have && in[i])
#pragma unroll
                    for (int m = 0; m < R; ++m) {
                        float y[V];
                        for (int k = 0; k < V; ++k)
                            y[k] = l == 0 ? fmaf(v[b][m][i][k], f[k], bias[i][k]) : v[b][m][i][k] * f[k];
                        store_vec<YT, V>(to, 0, y);
                        to += C * EY;
                    }
            }
            if (t == 0 && b < u.have) {
                const int64_t node = u.first + b * teams;
                if (l == 0 && a.mean) a.mean[node] = mu[b];
                if (a.rstd) a.rstd[node * (a.L + 1) + l] = q[b];
            }
        }
    }
}

template <int XT, int YT, int NI>
__global__ void __launch_bounds__(32 * kFwdWarps, 2) k_norm_teams(NormArgs a, int TL, Slots sl) {
    extern __shared__ __align__(16) char smem[];
    if (threadIdx.x < 16)
        reinterpret_cast<float*>(smem + (blockDim.x >> 5) * sl.stages * sl.stage_bytes)[threadIdx.x] = 0.f;
    __syncthreads();
    const int blk = blockIdx.x;
    if (blk < sl.at[1]) norm_degree<XT, YT, NI, 0>(a, TL, sl, smem);
    else if (blk < sl.at[2]) norm_degree<XT, YT, NI, 1>(a, TL, sl, smem);
    else if (blk < sl.at[3]) norm_degree<XT, YT, NI, 2>(a, TL, sl, smem);
    else if (blk < sl.at[4]) norm_degree<XT, YT, NI, 3>(a, TL, sl, smem);
    else norm_degree<XT, YT, NI, 4>(a, TL, sl, smem);
}

// One block per (node, degree), for L >= 1 with more than 256 channels: reads its
// group once per pass, from the second on out of L2. 4,000 atoms, L = 4, C = 260, fp32
// with a residual to bf16, 364 MB in 88 us.
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

// L = 0: one block per row, the row in registers, NV vectors of V values a thread.
// All of a row's loads are in flight together; rows of other blocks of the SM hide
// the two sums. 8,192 rows of 4,096 fp32 values with a residual, 470 MB in 71 us (the
// copy rate). TT > 0: that many threads, so that the offsets of a thread's values are
// constants; where V = 1 the instructions bound it (4,099 rows of 5,001 bf16 values:
// 42 us, 46 us without). V = 1 serves codes, rows with a checkpoint and the longest rows;
// the others run in k_norm_kept.
template <int XT, int YT, int V, int NV, int TT>
__global__ void __launch_bounds__(TT ? TT : 1024) k_norm_held(NormArgs a) {
    __shared__ float sh[32];
    const int64_t row = blockIdx.x, base = row * a.C + threadIdx.x * V;
    const int T = TT ? TT : blockDim.x, C = a.C - threadIdx.x * V;  // this thread's vector j exists: j T V < C
    const char* x = static_cast<const char*>(a.x) + base * (vec_bytes<XT>() / 4);
    float v[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        for (int k = 0; k < V; ++k) v[j][k] = 0.f;
        if (j * T * V < C) {
            if constexpr (XT == kMXI8)
                load_codes<V>(static_cast<const int8_t*>(a.x), a.xs, row, a.C, a.nb, (j * T + threadIdx.x) * V, v[j]);
            else
                load_vec<XT, V>(x, j * T * V, v[j]);
        }
    }
    if constexpr (XT != kMXI8) {
        if (a.res) {
            float r[NV][V];
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                for (int k = 0; k < V; ++k) r[j][k] = 0.f;
                if (j * T * V < C) load_vec<kF32, V>(a.res + base, j * T * V, r[j]);
            }
            char* sum = static_cast<char*>(a.sum) + base * (vec_bytes<XT>() / 4);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                for (int k = 0; k < V; ++k) v[j][k] = as_stored<XT>(v[j][k] + r[j][k]);
                if (j * T * V < C) store_vec<XT, V>(sum, j * T * V, v[j]);
            }
        }
        if (a.codes)
#pragma unroll
            for (int j = 0; j < NV; ++j)
                store_codes<V>(a.codes, a.scales, row, a.C, a.nb, (j * T + threadIdx.x) * V, j * T * V < C, 32, v[j]);
    }
    float s = 0.f, q = 0.f, w[NV][V], b[NV][V];  // the weights arrive while the sums are formed
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        for (int k = 0; k < V; ++k) w[j][k] = b[j][k] = 0.f;
        if (j * T * V < C) {
            load_vec<kF32, V>(a.w + threadIdx.x * V, j * T * V, w[j]);
            if (a.b) load_vec<kF32, V>(a.b + threadIdx.x * V, j * T * V, b[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
        for (int k = 0; k < V; ++k) s += v[j][k];
    const float mu = block_sum(s, sh) * a.inv_c;
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (j * T * V < C)
            for (int k = 0; k < V; ++k) {
                v[j][k] -= mu;
                q += v[j][k] * v[j][k];
            }
    const float r = rsqrtf(block_sum(q, sh) * a.inv_c + a.eps);
    char* y = static_cast<char*>(a.y) + base * (vec_bytes<YT>() / 4);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        for (int k = 0; k < V; ++k) v[j][k] = fmaf(v[j][k] * r, w[j][k], b[j][k]);
        if (j * T * V < C) store_vec<YT, V>(y, j * T * V, v[j]);
    }
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mu;
        if (a.rstd) a.rstd[row] = r;
    }
}

// A value as storage keeps it, so that its load can be under way while the one before it is in use.
template <int T>
struct Raw1 {
    float a;
    __device__ __forceinline__ void load(const char* p, int i) { a = reinterpret_cast<const float*>(p)[i]; }
    __device__ __forceinline__ float get() const { return a; }
};
template <>
struct Raw1<kBF16> {
    unsigned short a;
    __device__ __forceinline__ void load(const char* p, int i) { a = reinterpret_cast<const unsigned short*>(p)[i]; }
    __device__ __forceinline__ float get() const { return __uint_as_float((uint32_t)a << 16); }
};

// L = 0, fp32 or bf16 rows that no vector divides: persistent blocks, a thread's
// weights in registers from row to row, the next row's values under way while this
// one's sums are formed. Instructions bound it (one load, one store and about ten
// more a value). 4,099 rows of 5,001 bf16 values: 30 us (2.8 TB/s; one block per row
// 42 us), at 384 threads of 16 values (1,024 of 8: 37 us); 4,096 rows of 8,190: 43 us
// at 1,024 threads of 8 (512 of 16: 66 us); 20,000 rows of 1,001 fp32 values: 28 us
// (5.7 TB/s).
template <int XT, int YT, int NV, int TT>
__global__ void __launch_bounds__(TT) k_norm_kept(NormArgs a) {
    constexpr int E = vec_bytes<XT>() / 4, EY = vec_bytes<YT>() / 4;
    __shared__ float sh[2][32];
    const int C = a.C - threadIdx.x;  // this thread's value j exists: j TT < C
    float w[NV], b[NV];
    Raw1<XT> next[NV];
    auto load = [&](int64_t row) {
        const char* x = static_cast<const char*>(a.x) + (row * a.C + threadIdx.x) * E;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * TT < C) next[j].load(x, j * TT);
    };
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        w[j] = j * TT < C ? a.w[threadIdx.x + j * TT] : 0.f;
        b[j] = j * TT < C && a.b ? a.b[threadIdx.x + j * TT] : 0.f;
        next[j].a = 0;
    }
    if (blockIdx.x < a.n) load(blockIdx.x);
    for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
        const int64_t base = row * a.C + threadIdx.x;
        float v[NV], s = 0.f, q = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) v[j] = next[j].get();
        if (a.res)
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (j * TT < C) {
                    const float h[1] = {as_stored<XT>(v[j] + a.res[base + j * TT])};
                    v[j] = h[0];
                    store_vec<XT, 1>(static_cast<char*>(a.sum) + base * E, j * TT, h);
                }
        if (row + gridDim.x < a.n) load(row + gridDim.x);
#pragma unroll
        for (int j = 0; j < NV; ++j) s += v[j];  // values beyond the row are zero
        const float mu = block_sum(s, sh[0]) * a.inv_c;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            v[j] -= mu;
            if (j * TT < C) q = fmaf(v[j], v[j], q);
        }
        const float r = rsqrtf(block_sum(q, sh[1]) * a.inv_c + a.eps);
        char* y = static_cast<char*>(a.y) + base * EY;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const float o[1] = {fmaf(v[j] * r, w[j], b[j])};
            if (j * TT < C) store_vec<YT, 1>(y, j * TT, o);
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mu;
            if (a.rstd) a.rstd[row] = r;
        }
    }
}

template <int XT, int YT, int NV, int TT>
cudaError_t launch_kept(const NormArgs& a, cudaStream_t s) {
    // the blocks that fit at once: up to 64 registers a thread at NV = 8, 80 at 16 (97 from bf16 to fp32: 4,099 rows
    // of 5,001 values 36.0 us in one block an SM, 37.6 us in two)
    constexpr int per_sm = (NV == 8 ? 1024 : XT == kBF16 && YT == kF32 ? 384 : 768) / TT;
    k_norm_kept<XT, YT, NV, TT><<<(unsigned)std::min<int64_t>(a.n, kSMs * per_sm), TT, 0, s>>>(a);
    return cudaGetLastError();
}

template <int XT, int YT, int NI>
cudaError_t launch_teams(const NormArgs& a, const TeamPlan& p, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(k_norm_teams<XT, YT, NI>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBlockSmem);
    if (e != cudaSuccess) return e;
    Slots sl{p.stage_bytes, p.stages, kUnitRows * NI * 32 * vec_bytes<XT>(), 0, 0, {}};
    std::copy(p.at, p.at + kMaxL + 2, sl.at);
    k_norm_teams<XT, YT, NI><<<p.at[kMaxL + 1], 32 * p.warps, p.smem, s>>>(a, p.TL, sl);
    return cudaGetLastError();
}

template <int XT, int YT>
cudaError_t launch_fwd(const NormArgs& a, cudaStream_t s) {
    count_launch();
    if (use_teams(a.C)) {
        const int vec = vec_bytes<XT>() + (a.res ? 16 : 0);
        const TeamPlan p = team_plan(a.n, a.L, a.C, vec, vec, 0, kFwdWarps);
        return p.NI == 1 ? launch_teams<XT, YT, 1>(a, p, s) : launch_teams<XT, YT, 2>(a, p, s);
    }
    if (a.C <= kTeamC) return run_norm_scalar(a, XT, YT == kBF16, s);
    if (a.L == 0) {  // C <= 16384 always fits
        const unsigned grid = (unsigned)a.n;
        if (a.C % 4 == 0) k_norm_held<XT, YT, 4, 4, 0><<<grid, held_threads(a.C, 4, 4), 0, s>>>(a);
        else if (XT != kMXI8 && !a.codes && a.C <= 8192) {
            if constexpr (XT != kMXI8)
                return a.C <= 1024   ? launch_kept<XT, YT, 8, 128>(a, s)
                       : a.C <= 4096 ? launch_kept<XT, YT, 8, 512>(a, s)
                       : a.C <= 6144 ? launch_kept<XT, YT, 16, 384>(a, s)
                                     : launch_kept<XT, YT, 8, 1024>(a, s);
        } else if (a.C <= 1024) k_norm_held<XT, YT, 1, 8, 128><<<grid, 128, 0, s>>>(a);
        else if (a.C <= 6144) k_norm_held<XT, YT, 1, 16, 384><<<grid, 384, 0, s>>>(a);
        else k_norm_held<XT, YT, 1, 16, 1024><<<grid, 1024, 0, s>>>(a);
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
    NormArgs a{n_atoms, cfg->L, cfg->C, ck_blocks(cfg->C), cfg->eps, 1.f / cfg->C, x, x_scales, residual,
               sum,     weight, bias,   y,                 mean,     rstd, ck_codes, ck_scales};
    cudaStream_t s = static_cast<cudaStream_t>(stream_);
    const bool yb = cfg->y_dtype == E2F_BF16;
    E2F_CUDA_TRY(coded                       ? launch_fwd_y<kMXI8>(a, yb, s)
                 : cfg->x_dtype == E2F_BF16 ? launch_fwd_y<kBF16>(a, yb, s)
                                             : launch_fwd_y<kF32>(a, yb, s));
    return E2F_OK;
}
