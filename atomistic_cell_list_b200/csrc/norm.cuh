// Layer norm of irreducible features: what the forward (norm.cu) and the
// backward (norm_bwd.cu) share.
//
// Per node and degree l, over the group of (2l+1) rows of C channels:
//   d = h - mean_c h[0]  (l = 0),  d = h  (l >= 1);   r = 1/sqrt(mean d^2 + eps)
//   y = weight[l,c] d r  (+ bias[c] for l = 0)
// and with xh = d r, u = grad_y weight:
//   grad_x = r (u - xh mean(u xh)  [- mean u for l = 0]) (+ grad_skip)
//   grad_weight[l,c] = sum_{n,m} grad_y xh,   grad_bias[c] = sum_n grad_y[n,0,c]
// All sums are fp32, those of the weight's gradient in chains of a unit's rows, then of
// units. A few operations per value: memory bound.
//
// C a multiple of 4 up to 256 (the attention takes multiples of 16): a team of TL lanes (a
// power of two, TL >= C/4 up to 32) owns whole rows, lane t the channels
// 4 (t + TL i) .. +3, i < NI. A block works on one degree, so that its code has the
// rows of a group unrolled and stays in the instruction cache (with all degrees in
// every block the warps waited for instructions; with one code for all degrees
// they executed twice as many). One warp takes a unit: as many nodes per team as
// make 5 to 9 rows, held in registers. A (node, degree) group is contiguous in
// memory: its team copies it in 16-byte pieces (cp.async) to the warp's own part of
// shared memory, one to three units ahead of the one in work. Warps never wait for
// one another, and the bytes in flight (about 100 KB an SM) do not depend on
// registers or occupancy. Lanes beyond the row read zeros.
// Other C up to 256: one warp per unit, values one by one (norm_scalar.cu).
// L = 0 with more channels: a block per row, or persistent blocks that go from row to
// row, the row in registers. The rest: one block per (node, degree), which reads its
// group once per pass.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "feature_io.cuh"

namespace e2f {
struct NormArgs {
    int64_t n;
    int L, C, nb;
    float eps, inv_c;
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
    float inv_c;
    const void* x;
    const uint8_t* xs;
    const float* w;
    const float* mean;
    const float* rstd;
    const float* gy;
    const float* skip;
    float* gx;
    float* part;  // weight-gradient partials (null: not wanted)
    int g;        // k_norm_bwd_rows: degree l has g (2l+1) blocks
};

// up to 256 channels, any number: norm_scalar.cu. at: the blocks of degree l are [at[l], at[l+1]), at[0] = 0.
cudaError_t run_norm_scalar(const NormArgs& a, int x_type, bool y_bf16, cudaStream_t s);
cudaError_t run_norm_bwd_scalar(const NormBwdArgs& a, int x_type, int* at, cudaStream_t s);

namespace {

constexpr int kMaxNormC = 16384;
constexpr int kNormBlocks = 592;  // most blocks of a weight-gradient pass: 4 on each of 148 SMs

constexpr int kSMs = 148;
constexpr int kTeamC = 256;  // most channels a team holds

constexpr int kUnitRows = 9;  // most rows of a unit per team
constexpr int kBlockSmem = 113 * 1024;  // two blocks per SM
constexpr int kTeamBlocks = 2 * kSMs;

// nodes of degree l that a team takes at once
__host__ __device__ constexpr int unit_nodes(int l) { return l == 0 ? 9 : l == 1 ? 3 : 1; }

// The blocks [at[l], at[l+1]) work on degree l.
struct TeamPlan {
    int NI, TL, warps, stages, stage_bytes;  // stages: units per warp in flight or in work
    int at[kMaxL + 2];
    size_t smem;
};

// where the second and third stream and the statistics of a unit lie in a stage
struct Slots {
    int stage_bytes, stages, o1, o2, o3, at[kMaxL + 2];
};

bool use_teams(int C) { return C % 4 == 0 && C <= kTeamC; }

// bytes of 4 channels
template <int T>
constexpr int vec_bytes() { return T == kF32 ? 16 : T == kBF16 ? 8 : 4; }

// Plan of n nodes whose units read `vec` bytes per lane and vector of 4 channels
// (`most` with every optional input) and `small` more bytes per stage. As many
// warps as a block's shared memory gives two stages of `most`, up to `cap` (by
// registers), then up to 4 stages: which warp takes which unit, and so the order of
// the weight gradient's sums, does not depend on the optional inputs. Degrees get
// blocks by their rows, with half a row more for a group's sums.
TeamPlan team_plan(int64_t n, int L, int C, int vec, int most, int small, int cap) {
    TeamPlan p{};
    p.TL = 4;
    while (p.TL < 32 && p.TL * 4 < C) p.TL *= 2;
    p.NI = p.TL * 4 < C ? 2 : 1;
    const int row = kUnitRows * p.NI * 32;
    p.stage_bytes = row * vec + small;
    p.warps = std::min(cap, (kBlockSmem - 64) / (2 * (row * most + small)));
    p.stages = std::min(4, (kBlockSmem - 64) / p.warps / p.stage_bytes);
    p.smem = (size_t)p.warps * p.stages * p.stage_bytes + 64;
    const double rows = (L + 1) * (L + 1) + 0.5 * (L + 1);
    for (int l = 0; l <= L; ++l) {
        const int64_t units = (n + unit_nodes(l) * (32 / p.TL) - 1) / (unit_nodes(l) * (32 / p.TL));
        const int share = std::max(1, (int)(kTeamBlocks * (2 * l + 1.5) / rows));
        p.at[l + 1] = p.at[l] + (int)std::min<int64_t>(share, units);
    }
    for (int l = L + 1; l <= kMaxL; ++l) p.at[l + 1] = p.at[l];
    return p;
}

__device__ __forceinline__ void cp_async16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
template <int BYTES>  // 4 or 8
__device__ __forceinline__ void cp_async_small(uint32_t to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the newest n groups of this thread have arrived
__device__ __forceinline__ void cp_wait(int n) {
    if (n <= 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else if (n == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else asm volatile("cp.async.wait_group 3;" ::: "memory");
}

// A lane's view of unit k of degree l, B nodes per team: first, first + teams, ...
template <int NI, int l>
struct Unit {
    static constexpr int R = 2 * l + 1, B = unit_nodes(l);
    int64_t first, row0;
    int have;  // node b exists: b < have
    __device__ __forceinline__ Unit(int64_t k, int64_t n, int K, int TL) {
        const int teams = 32 / TL;
        first = k * (B * teams) + (threadIdx.x & 31) / TL;
        row0 = first * K + l * l;
        const int64_t left = n - first;
        have = left <= 0 ? 0 : left >= B * teams ? B : (int)(left + teams - 1) / teams;
    }
    // starts the copies of one stream [rows, C] of storage T to `to`: [team][node][row][C],
    // in 16-byte pieces, or vector by vector where rows do not begin on 16 bytes
    template <int T>
    __device__ __forceinline__ void fetch(const void* p, int C, int K, int TL, uint32_t to) const {
        constexpr int IT = (R * NI * vec_bytes<T>() + 15) / 16;
        const int lane = threadIdx.x & 31, t16 = (lane & (TL - 1)) * 16, bytes = R * C * (vec_bytes<T>() / 4);
        const char* q = static_cast<const char*>(p) + row0 * C * (vec_bytes<T>() / 4) + t16;
        to += lane / TL * (B * bytes) + t16;
        if constexpr (T != kF32)
            if (C * (vec_bytes<T>() / 4) % 16) {
                constexpr int VB = vec_bytes<T>();
                const int t = lane & (TL - 1);
                q += t * VB - t16;
                to += t * VB - t16;
                for (int b = 0; b < have; ++b) {
                    for (int o = 0; o < R; ++o)
#pragma unroll
                        for (int i = 0; i < NI; ++i)
                            if ((t + TL * i) * 4 < C)
                                cp_async_small<VB>(to + (o * (C / 4) + TL * i) * VB, q + (o * (C / 4) + TL * i) * VB);
                    q += (int64_t)(32 / TL * K) * C * (VB / 4);
                    to += bytes;
                }
                return;
            }
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (b < have) {
#pragma unroll
                for (int j = 0; j < IT; ++j)
                    if (t16 + j * TL * 16 < bytes) cp_async16(to + (b * bytes + j * TL * 16), q + j * TL * 16);
                q += (int64_t)(32 / TL * K) * C * (vec_bytes<T>() / 4);
            }
    }
    // scale bytes of a checkpoint's vectors, one lane's
    __device__ __forceinline__ void scales(const uint8_t* xs, int nb, int K, int TL, const int (&c)[NI],
                                           uint32_t (&s)[B * R][NI]) const {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const uint8_t* q = xs + row0 * nb + c[i] / kCkBlock;
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const uint8_t* p = q;
                if (b < have)
#pragma unroll
                    for (int m = 0; m < R; ++m, p += nb) s[b * R + m][i] = *p;
                q += (int64_t)(32 / TL * K) * nb;
            }
        }
    }
};

template <int N>
__device__ __forceinline__ void team_sum(float (&v)[N], int TL) {
    for (int o = TL >> 1; o; o >>= 1)
#pragma unroll
        for (int b = 0; b < N; ++b) v[b] += __shfl_xor_sync(0xffffffffu, v[b], o);
}

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

// threads for rows of C values held in registers, nv vectors of v each; 0: the row is too long
int held_threads(int C, int v, int nv, int most = 1024) {
    const int t = ((C + v * nv - 1) / (v * nv) + 31) / 32 * 32;
    return t <= most ? t : 0;
}

int row_threads(int C, int V) {
    int t = 32;
    while (t < 512 && t * V < C) t *= 2;
    return t;
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
