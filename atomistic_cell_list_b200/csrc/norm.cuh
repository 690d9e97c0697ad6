// Layer norm of irreducible features: what the forward (norm.cu) and the
// backward (norm_bwd.cu) share.
//
// Per node and degree l, over the group of (2l+1) rows of C channels:
//   d = h - mean_c h[0]  (l = 0),  d = h  (l >= 1);   r = 1/sqrt(mean d^2 + eps)
//   y = weight[l,c] d r  (+ bias[c] for l = 0)
// and with xh = d r, u = grad_y weight:
//   grad_x = r (u - xh mean(u xh)  [- mean u for l = 0]) (+ grad_skip)
//   grad_weight[l,c] = sum_{n,m} grad_y xh,   grad_bias[c] = sum_n grad_y[n,0,c]
// All sums are fp32. A few operations per value: memory bound.
//
// C a multiple of 4 up to 256: a team of lanes per row, everything in
// registers, one pass over the data. A team of TL lanes (a power of two,
// TL >= C/4 up to 32) owns whole rows: lane t holds channels 4 (t + TL i) .. +3,
// i < NI, of all 2l+1 rows of a group, and of B nodes at once where groups are
// small, so that 6 to 10 row loads are in flight per lane at every degree
// (NI = 1). Sums are shuffles. Chunks of S nodes with all their degrees keep a
// chunk's rows close in time and in address.
// Any other C: one block per (node, degree).
#pragma once

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
    int g;        // k_norm_bwd_rows: degree l has g (2l+1) blocks
};

constexpr int kSMs = 148;
constexpr int kTeamC = 256;  // most channels a team holds

// nodes of degree l that a team takes at once, to have about `rows` rows in its registers
constexpr int nodes_of(int l, int rows) { return rows / (2 * l + 1) < 1 ? 1 : rows / (2 * l + 1); }
// the backward holds x and grad_y: fewer rows, within 128 registers at NI = 1
constexpr int fwd_rows(int NI) { return NI == 1 ? 9 : 5; }
constexpr int bwd_rows(int NI) { return NI == 1 ? 6 : 3; }

struct Units {  // units (one warp, one degree, B nodes per team) of a chunk of S nodes
    int n[kMaxL + 1], total;
};

struct TeamPlan {
    int NI, TL, S;
    int64_t chunks;
    Units un;
};

bool use_teams(int C) { return C % 4 == 0 && C <= kTeamC; }

// Lanes and chunk size for n nodes: chunks of 24 nodes a team (whole units at
// every degree), fewer when that gives less than `blocks` chunks.
TeamPlan team_plan(int64_t n, int L, int C, int blocks, bool fwd) {
    TeamPlan p{};
    p.TL = 1;
    while (p.TL < 32 && p.TL * 4 < C) p.TL *= 2;
    p.NI = p.TL * 4 < C ? 2 : 1;
    const int teams = 32 / p.TL;
    p.S = 24 * teams;
    while (p.S > 1 && (n + p.S - 1) / p.S < blocks) p.S = (p.S + 1) / 2;
    p.chunks = (n + p.S - 1) / p.S;
    for (int l = 0; l <= L; ++l) {
        const int per = nodes_of(l, fwd ? fwd_rows(p.NI) : bwd_rows(p.NI)) * teams;
        p.un.n[l] = (p.S + per - 1) / per;
        p.un.total += p.un.n[l];
    }
    return p;
}

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
