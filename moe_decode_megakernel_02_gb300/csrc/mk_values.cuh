// mk_values.cuh -- values of rows in the caller's memory, eight at a time:
// loaded as they lie there, seen as 32-bit numbers, stored rounded once.
#pragma once
#include "mk_ops.cuh"

namespace mkop {

// the larger of magnitudes (of one 32-bit number, or of two 16-bit ones); NaN wins
template <int DT>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    if constexpr (DT == MK_DT_F32) return max(a, b);
    uint32_t y;
    if constexpr (DT == MK_DT_BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}

// Eight values of a row outside the cache, as they lie there. VEC: 16-byte
// aligned.
template <int DT, bool VEC>
struct Values8 {
    static constexpr int W = DT == MK_DT_F32 ? 8 : 4;  // 32-bit words
    uint32_t w[W];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void load(const uint8_t* base, long long at) {
        if constexpr (VEC) {
            const uint4* p = reinterpret_cast<const uint4*>(base + at * (DT == MK_DT_F32 ? 4 : 2));
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
                const uint4 a = __ldcs(p + i);
                w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
            }
        } else if constexpr (DT == MK_DT_F32) {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(base) + at;
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = p[i];
        } else {
            const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + at;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
        }
    }
    // 16-bit types are exact in 32 bits
    __device__ __forceinline__ void floats(float (&x)[8]) const {
        if constexpr (DT == MK_DT_F32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DT == MK_DT_BF16) {
                    x[2 * i] = __uint_as_float(w[i] << 16);
                    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                } else {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                    x[2 * i] = f.x;
                    x[2 * i + 1] = f.y;
                }
            }
        }
    }
    // the largest magnitude's bits; 16-bit types: of the even and of the odd values, side by side
    __device__ __forceinline__ uint32_t largest() const {
        constexpr uint32_t ABS = DT == MK_DT_F32 ? 0x7fffffffu : 0x7fff7fffu;
        uint32_t m = w[0] & ABS;
#pragma unroll
        for (int i = 1; i < W; ++i) m = larger<DT>(m, w[i] & ABS);
        return m;
    }
};
template <int DT, bool VEC>
__device__ __forceinline__ void store8(uint8_t* base, long long at, const float (&x)[8]) {
    if constexpr (DT == MK_DT_F32) {
        float* p = reinterpret_cast<float*>(base) + at;
        if constexpr (VEC) {
            __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
            __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = x[i];
        }
    } else {
        uint16_t* p = reinterpret_cast<uint16_t*>(base) + at;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = DT == MK_DT_BF16 ? pack_bf16(x[2 * i], x[2 * i + 1]) : pack_f16(x[2 * i], x[2 * i + 1]);
        if constexpr (VEC) {
            __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[2 * i] = (uint16_t)w[i];
                p[2 * i + 1] = (uint16_t)(w[i] >> 16);
            }
        }
    }
}

}  // namespace mkop
