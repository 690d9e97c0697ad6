// 8-bit activation checkpoints: blocks of 32 channels of one row share a power
// of two 2^e, e = floor(log2 max |x|); a value is kept as the whole number
// rint(x 2^(6-e)) in 8 bits (feature_io.cuh). One pass over the data; memory
// bound.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"
#include "feature_io.cuh"

namespace e2f {
namespace {

unsigned ck_grid(int64_t threads) { return (unsigned)std::min<int64_t>((threads + 255) / 256, 148 * 64); }

// C a multiple of 32: rows need no attention, the tensor is a run of blocks of 32
// values. A thread takes 8 values, four threads a block, U vectors of a thread are
// in flight. 30,000 atoms, L = 4, C = 128 in bf16: store 50 us, load 42 us, 291 MB
// each (6.3 TB/s together; 4 values a thread, found by divisions, took 219 us).
constexpr int kFlat = 8, kU = 4;

template <int T>
__global__ void __launch_bounds__(256) k_ck_store_flat(const void* x, int64_t vecs, int8_t* codes, uint8_t* scales) {
    const int64_t first = (int64_t)blockIdx.x * (256 * kU) + threadIdx.x;
    float v[kU][kFlat];
#pragma unroll
    for (int u = 0; u < kU; ++u)
        if (first + u * 256 < vecs) load8<T>(x, first + u * 256, v[u]);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const int64_t i = first + u * 256;
        float m = fabsf(v[u][0]);
#pragma unroll
        for (int k = 1; k < kFlat; ++k) m = mag_max(m, v[u][k]);
        m = mag_max(m, __shfl_xor_sync(0xffffffffu, m, 1));  // vecs is a multiple of 4: a block's lanes exist together
        m = mag_max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        if (i >= vecs) continue;
        const uint32_t s = ck_byte(m);
        const float inv = ck_inverse(s);
        uint2 q;
        q.x = pack_codes(v[u][0], v[u][1], v[u][2], v[u][3], inv);
        q.y = pack_codes(v[u][4], v[u][5], v[u][6], v[u][7], inv);
        if (s == 255u) q = make_uint2(0u, 0u);
        reinterpret_cast<uint2*>(codes)[i] = q;
        if ((i & 3) == 0) scales[i >> 2] = (uint8_t)s;
    }
}

template <int T>
__global__ void __launch_bounds__(256) k_ck_load_flat(const int8_t* codes, const uint8_t* scales, int64_t vecs,
                                                      void* out) {
    const int64_t first = (int64_t)blockIdx.x * (256 * kU) + threadIdx.x;
    uint2 q[kU];
    uint32_t s[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u)
        if (first + u * 256 < vecs) {
            q[u] = reinterpret_cast<const uint2*>(codes)[first + u * 256];
            s[u] = scales[(first + u * 256) >> 2];
        }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        if (first + u * 256 >= vecs) continue;
        Raw4<kMXI8> r;
        float v[kFlat], w[4];
        r.s = s[u];
        r.a = q[u].x;
        r.get(w);
        for (int k = 0; k < 4; ++k) v[k] = w[k];
        r.a = q[u].y;
        r.get(w);
        for (int k = 0; k < 4; ++k) v[4 + k] = w[k];
        store8<T>(out, first + u * 256, v);
    }
}

// any C: 32/V lanes per block of channels, found by divisions. 30,000 atoms, L = 4, bf16,
// store and load together: C = 100 (228 MB a way) 161 us, C = 101, value by value, 556 us.
template <int T, int V>
__global__ void __launch_bounds__(256) k_ck_store(const void* x, int64_t rows, int C, int nb, int8_t* codes,
                                                  uint8_t* scales) {
    constexpr int G = kCkBlock / V;
    const int64_t total = rows * nb * G, step = (int64_t)gridDim.x * 256;
    for (int64_t i0 = blockIdx.x * 256ll; i0 < total; i0 += step) {
        const int64_t i = i0 + threadIdx.x, blk = i / G, row = blk / nb;
        const int c = (int)(blk - row * nb) * kCkBlock + (int)(i % G) * V;
        const bool ok = i < total && c < C;
        float v[V] = {};
        if (ok) load_vec<T, V>(x, row * C + c, v);
        store_codes<V>(codes, scales, row, C, nb, c, ok, 32, v);
    }
}

template <int T, int V>
__global__ void __launch_bounds__(256) k_ck_load(const int8_t* codes, const uint8_t* scales, int64_t rows, int C,
                                                 int nb, void* out) {
    const int cv = C / V;
    const int64_t total = rows * cv, step = (int64_t)gridDim.x * 256;
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += step) {
        const int64_t row = i / cv;
        const int c = (int)(i - row * cv) * V;
        float v[V];
        load_codes<V>(codes, scales, row, C, nb, c, v);
        store_vec<T, V>(out, row * C + c, v);
    }
}

template <int T>
cudaError_t launch_store(const void* x, int64_t rows, int C, int8_t* codes, uint8_t* scales, cudaStream_t s) {
    const int nb = ck_blocks(C);
    const int64_t vecs = rows * (C / kFlat), flat = (vecs + 256 * kU - 1) / (256 * kU);
    count_launch();
    if (C % kCkBlock == 0 && flat <= INT32_MAX)
        k_ck_store_flat<T><<<(unsigned)flat, 256, 0, s>>>(x, vecs, codes, scales);
    else if (C % 4 == 0)
        k_ck_store<T, 4><<<ck_grid(rows * nb * 8), 256, 0, s>>>(x, rows, C, nb, codes, scales);
    else
        k_ck_store<T, 1><<<ck_grid(rows * nb * 32), 256, 0, s>>>(x, rows, C, nb, codes, scales);
    return cudaGetLastError();
}

template <int T>
cudaError_t launch_load(const int8_t* codes, const uint8_t* scales, int64_t rows, int C, void* out, cudaStream_t s) {
    const int nb = ck_blocks(C);
    const int64_t vecs = rows * (C / kFlat), flat = (vecs + 256 * kU - 1) / (256 * kU);
    count_launch();
    if (C % kCkBlock == 0 && flat <= INT32_MAX)
        k_ck_load_flat<T><<<(unsigned)flat, 256, 0, s>>>(codes, scales, vecs, out);
    else if (C % 4 == 0)
        k_ck_load<T, 4><<<ck_grid(rows * (C / 4)), 256, 0, s>>>(codes, scales, rows, C, nb, out);
    else
        k_ck_load<T, 1><<<ck_grid(rows * C), 256, 0, s>>>(codes, scales, rows, C, nb, out);
    return cudaGetLastError();
}

e2f_status check_ck(const void* x, e2f_dtype dtype, int64_t rows, int C, const void* codes, const void* scales) {
    if (rows < 0 || C <= 0) return E2F_ERR_INVALID_ARG;
    if (dtype != E2F_F32 && dtype != E2F_BF16) return E2F_ERR_UNSUPPORTED;
    if (rows > INT64_MAX / 8 / C) return E2F_ERR_INVALID_ARG;
    if (rows == 0) return E2F_OK;
    if (!x || !codes || !scales) return E2F_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(x) % 16 || reinterpret_cast<uintptr_t>(codes) % 16) return E2F_ERR_ALIGNMENT;
    return E2F_OK;
}

}  // namespace
}  // namespace e2f

using namespace e2f;

extern "C" e2f_status e2f_checkpoint_store(const void* x, e2f_dtype dtype, int64_t rows, int C, int8_t* codes,
                                           uint8_t* scales, void* stream) {
    e2f_status st = check_ck(x, dtype, rows, C, codes, scales);
    if (st != E2F_OK || rows == 0) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    E2F_CUDA_TRY(dtype == E2F_F32 ? launch_store<kF32>(x, rows, C, codes, scales, s)
                                  : launch_store<kBF16>(x, rows, C, codes, scales, s));
    return E2F_OK;
}

extern "C" e2f_status e2f_checkpoint_load(const int8_t* codes, const uint8_t* scales, int64_t rows, int C,
                                          e2f_dtype dtype, void* out, void* stream) {
    e2f_status st = check_ck(out, dtype, rows, C, codes, scales);
    if (st != E2F_OK || rows == 0) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    E2F_CUDA_TRY(dtype == E2F_F32 ? launch_load<kF32>(codes, scales, rows, C, out, s)
                                  : launch_load<kBF16>(codes, scales, rows, C, out, s));
    return E2F_OK;
}
