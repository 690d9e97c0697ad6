// Vector loads and stores of node features (fp32, bf16 or 8-bit checkpoint)
// and the checkpoint's block format, shared by the norm, embedding and
// checkpoint kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace e2f {

constexpr int kCkBlock = 32;  // channels that share one scale byte
__host__ __device__ inline int ck_blocks(int C) { return (C + kCkBlock - 1) / kCkBlock; }

enum { kF32 = 0, kBF16 = 1, kMXI8 = 2 };  // e2f_dtype values, as template arguments

// V consecutive values of an fp32 or bf16 array (V = 4: address 4-value aligned)
template <int T, int V>
__device__ __forceinline__ void load_vec(const void* p, int64_t i, float (&v)[V]) {
    if constexpr (T == kF32) {
        const float* q = static_cast<const float*>(p) + i;
        if constexpr (V == 4) {
            const float4 a = *reinterpret_cast<const float4*>(q);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        } else {
            for (int k = 0; k < V; ++k) v[k] = q[k];
        }
    } else {
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p) + i;
        if constexpr (V == 4) {
            const uint2 a = *reinterpret_cast<const uint2*>(q);
            v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xffff0000u);
            v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xffff0000u);
        } else {
            for (int k = 0; k < V; ++k) v[k] = __bfloat162float(q[k]);
        }
    }
}

template <int T, int V>
__device__ __forceinline__ void store_vec(void* p, int64_t i, const float (&v)[V]) {
    if constexpr (T == kF32) {
        float* q = static_cast<float*>(p) + i;
        if constexpr (V == 4) {
            *reinterpret_cast<float4*>(q) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
            for (int k = 0; k < V; ++k) q[k] = v[k];
        }
    } else {
        __nv_bfloat16* q = static_cast<__nv_bfloat16*>(p) + i;
        if constexpr (V == 4) {
            __nv_bfloat162 a[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
            *reinterpret_cast<uint2*>(q) = *reinterpret_cast<uint2*>(a);
        } else {
            for (int k = 0; k < V; ++k) q[k] = __float2bfloat16_rn(v[k]);
        }
    }
}

// vector i of 8 consecutive values (16-byte aligned)
template <int T>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
    if constexpr (T == kF32) {
        const float4 a = static_cast<const float4*>(p)[2 * i], b = static_cast<const float4*>(p)[2 * i + 1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 a = static_cast<const uint4*>(p)[i];
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = __uint_as_float(w[k] << 16);
            v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
    }
}

template <int T>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
    if constexpr (T == kF32) {
        static_cast<float4*>(p)[2 * i] = make_float4(v[0], v[1], v[2], v[3]);
        static_cast<float4*>(p)[2 * i + 1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        __nv_bfloat162 a[4];
        for (int k = 0; k < 4; ++k) a[k] = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        static_cast<uint4*>(p)[i] = *reinterpret_cast<uint4*>(a);
    }
}

// fp32 value as storage type T keeps it
template <int T>
__device__ __forceinline__ float as_stored(float v) {
    if constexpr (T == kBF16) return __bfloat162float(__float2bfloat16_rn(v));
    return v;
}

// 2^(s - 127) for a scale byte; 255 marks a block that held a NaN or an infinity
__device__ __forceinline__ float ck_scale(uint32_t s) {
    return __uint_as_float(s == 255u ? 0x7fc00000u : s == 0u ? 0x00400000u : s << 23);
}

// scale byte of a block from its largest magnitude (NaN if any value is): the
// exponent of the largest value, at least 2^-120 so that the unit 2^(e-6) and
// its inverse are normal numbers
__device__ __forceinline__ uint32_t ck_byte(float top) { return max(__float_as_uint(top) >> 23, 7u); }

// the larger magnitude; a NaN on either side stays
__device__ __forceinline__ float mag_max(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}

// the unit 2^(s - 133) of a block, exact (at least 2^-133)
__device__ __forceinline__ float ck_unit(uint32_t s) {
    return s - 7u <= 247u ? __uint_as_float((s - 6u) << 23) : ck_scale(s) * 0.015625f;
}

// code of v in a block of scale byte s < 255: rint(v 2^(6-e)) clamped to +-127,
// in the low byte. The scaling is a power of two and fma rounds once, to whole
// numbers at 1.5 2^23 (half to even): the code does not depend on how it is computed.
__device__ __forceinline__ uint32_t ck_code(float v, float inv) {
    constexpr float kMagic = 12582912.f;
    return __float_as_uint(fminf(fmaxf(fmaf(v, inv, kMagic), kMagic - 127.f), kMagic + 127.f));
}
__device__ __forceinline__ float ck_inverse(uint32_t s) { return __uint_as_float((260u - s) << 23); }

// codes of four values, first in the low byte
__device__ __forceinline__ uint32_t pack_codes(float a, float b, float c, float d, float inv) {
    const uint32_t lo = __byte_perm(ck_code(a, inv), ck_code(b, inv), 0x0040);
    const uint32_t hi = __byte_perm(ck_code(c, inv), ck_code(d, inv), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}

// A code as fp32, without a conversion instruction: the byte with its sign bit
// turned over is code + 128, placed (by a byte permutation) in the low mantissa of 2^23.
__device__ __forceinline__ float ck_value(uint32_t biased, uint32_t select) {
    return __uint_as_float(__byte_perm(biased, 0x4b000000u, select)) - 8388736.f;
}

// Four channels as storage keeps them, so that loads can be issued in a batch
// before any value is used.
template <int T>
struct Raw4;
template <>
struct Raw4<kF32> {
    float4 a;
    // from shared memory, by its 32-bit address
    __device__ __forceinline__ void from(uint32_t p) {
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(a.x), "=f"(a.y), "=f"(a.z), "=f"(a.w) : "r"(p));
    }
    __device__ __forceinline__ void get(float (&v)[4]) const {
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    }
};
template <>
struct Raw4<kBF16> {
    uint2 a;
    __device__ __forceinline__ void from(uint32_t p) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(a.x), "=r"(a.y) : "r"(p));
    }
    __device__ __forceinline__ void get(float (&v)[4]) const {
        v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xffff0000u);
        v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xffff0000u);
    }
};
template <>
struct Raw4<kMXI8> {
    uint32_t a, s;
    __device__ __forceinline__ void from(uint32_t p) { asm volatile("ld.shared.u32 %0, [%1];" : "=r"(a) : "r"(p)); }
    __device__ __forceinline__ void load(const void* p, const uint8_t* scales, int64_t i, int64_t block) {
        a = *reinterpret_cast<const uint32_t*>(static_cast<const int8_t*>(p) + i);
        s = scales[block];
    }
    __device__ __forceinline__ void get(float (&v)[4]) const {
        const float u = ck_unit(s);
        const uint32_t b = a ^ 0x80808080u;
        v[0] = ck_value(b, 0x7650) * u; v[1] = ck_value(b, 0x7651) * u;
        v[2] = ck_value(b, 0x7652) * u; v[3] = ck_value(b, 0x7653) * u;
    }
};

// V decoded channels c .. c+V-1 of row `row` of a checkpoint (V = 4: c a multiple of 4, codes 4-byte aligned)
template <int V>
__device__ __forceinline__ void load_codes(const int8_t* codes, const uint8_t* scales, int64_t row, int C, int nb,
                                           int c, float (&v)[V]) {
    if constexpr (V == 4) {
        Raw4<kMXI8> r;
        r.load(codes, scales, row * C + c, row * nb + c / kCkBlock);
        r.get(v);
    } else {
        const float u = ck_unit(scales[row * nb + c / kCkBlock]);
        for (int k = 0; k < V; ++k) v[k] = codes[row * C + c + k] * u;
    }
}

// features of any storage: fp32, bf16, or a checkpoint (codes at p, scales at s)
template <int T, int V>
__device__ __forceinline__ void load_feat(const void* p, const uint8_t* s, int64_t row, int C, int nb, int c,
                                          float (&v)[V]) {
    if constexpr (T == kMXI8) {
        load_codes<V>(static_cast<const int8_t*>(p), s, row, C, nb, c, v);
    } else {
        load_vec<T, V>(p, row * C + c, v);
    }
}

// Checkpoint of V channels per lane, lanes in channel order: a block of 32
// channels is 32/V lanes, fewer when the lanes of a row (`team`) are fewer.
// Every lane of the warp calls it; lanes beyond the row pass zeros and ok = false.
// at: where this lane's codes go; scale: where its block's byte goes, written by the block's first lane.
template <int V>
__device__ __forceinline__ void store_codes_at(int8_t* at, uint8_t* scale, bool first, bool ok, int team,
                                               const float (&v)[V]) {
    float m = fabsf(v[0]);
    for (int k = 1; k < V; ++k) m = mag_max(m, v[k]);
    constexpr int G = kCkBlock / V;
    for (int o = 1; o < G; o <<= 1)
        if (o < team) m = mag_max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (!ok) return;
    const uint32_t s = ck_byte(m);
    const float inv = ck_inverse(s);
    if constexpr (V == 4) {
        *reinterpret_cast<uint32_t*>(at) = s == 255u ? 0u : pack_codes(v[0], v[1], v[2], v[3], inv);
    } else {
        for (int k = 0; k < V; ++k) at[k] = s == 255u ? 0 : (int8_t)ck_code(v[k], inv);
    }
    if (first) *scale = (uint8_t)s;
}

template <int V>
__device__ __forceinline__ void store_codes(int8_t* codes, uint8_t* scales, int64_t row, int C, int nb, int c, bool ok,
                                            int team, const float (&v)[V]) {
    store_codes_at<V>(codes + row * C + c, scales + row * nb + c / kCkBlock, c % kCkBlock == 0, ok, team, v);
}

}  // namespace e2f
