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

// 32/V lanes per block of channels
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

e2f_status check_ck(const void* x, e2f_dtype dtype, int64_t rows, int C, const void* codes, const void* scales) {
    if (rows < 0 || C <= 0) return E2F_ERR_INVALID_ARG;
    if (dtype != E2F_F32 && dtype != E2F_BF16) return E2F_ERR_UNSUPPORTED;
    if (rows > INT64_MAX / 8 / C) return E2F_ERR_INVALID_ARG;
    if (rows == 0) return E2F_OK;
    if (!x || !codes || !scales) return E2F_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(x) % 16 || reinterpret_cast<uintptr_t>(codes) % 16) return E2F_ERR_ALIGNMENT;
    return E2F_OK;
}

unsigned ck_grid(int64_t threads) { return (unsigned)std::min<int64_t>((threads + 255) / 256, 148 * 64); }

}  // namespace
}  // namespace e2f

using namespace e2f;

extern "C" e2f_status e2f_checkpoint_store(const void* x, e2f_dtype dtype, int64_t rows, int C, int8_t* codes,
                                           uint8_t* scales, void* stream) {
    e2f_status st = check_ck(x, dtype, rows, C, codes, scales);
    if (st != E2F_OK || rows == 0) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int nb = ck_blocks(C);
    count_launch();
    if (C % 4 == 0) {
        const unsigned g = ck_grid(rows * nb * 8);
        if (dtype == E2F_F32) k_ck_store<kF32, 4><<<g, 256, 0, s>>>(x, rows, C, nb, codes, scales);
        else k_ck_store<kBF16, 4><<<g, 256, 0, s>>>(x, rows, C, nb, codes, scales);
    } else {
        const unsigned g = ck_grid(rows * nb * 32);
        if (dtype == E2F_F32) k_ck_store<kF32, 1><<<g, 256, 0, s>>>(x, rows, C, nb, codes, scales);
        else k_ck_store<kBF16, 1><<<g, 256, 0, s>>>(x, rows, C, nb, codes, scales);
    }
    E2F_CUDA_TRY(cudaGetLastError());
    return E2F_OK;
}

extern "C" e2f_status e2f_checkpoint_load(const int8_t* codes, const uint8_t* scales, int64_t rows, int C,
                                          e2f_dtype dtype, void* out, void* stream) {
    e2f_status st = check_ck(out, dtype, rows, C, codes, scales);
    if (st != E2F_OK || rows == 0) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int nb = ck_blocks(C);
    count_launch();
    if (C % 4 == 0) {
        const unsigned g = ck_grid(rows * (C / 4));
        if (dtype == E2F_F32) k_ck_load<kF32, 4><<<g, 256, 0, s>>>(codes, scales, rows, C, nb, out);
        else k_ck_load<kBF16, 4><<<g, 256, 0, s>>>(codes, scales, rows, C, nb, out);
    } else {
        const unsigned g = ck_grid(rows * C);
        if (dtype == E2F_F32) k_ck_load<kF32, 1><<<g, 256, 0, s>>>(codes, scales, rows, C, nb, out);
        else k_ck_load<kBF16, 1><<<g, 256, 0, s>>>(codes, scales, rows, C, nb, out);
    }
    E2F_CUDA_TRY(cudaGetLastError());
    return E2F_OK;
}
