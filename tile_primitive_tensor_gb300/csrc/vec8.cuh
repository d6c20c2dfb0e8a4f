// Eight neighbouring elements at a time: conversions between a type's packed
// form and 32-bit values, and loads and stores of whole or partial groups.
#pragma once

#include <type_traits>

#include "elem.cuh"

namespace tpg {

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, __half>::value) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = p.x;
            f[2 * i + 1] = p.y;
        } else {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, __half>::value) {
            const __half2 p = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
        } else {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight 8-bit codes: nearest even, saturating.
__device__ __forceinline__ uint2 pack8_fp8(const float (&f)[8], __nv_fp8_interpretation_t kind) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, kind);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// The n (at most 8) elements at base[at]: one or two 16-byte accesses when
// `vec` (all eight, aligned), else one by one; the rest read as zero.
template <typename T>
__device__ __forceinline__ void load8(const void* base, int64_t at, bool vec, int n, float (&f)[8]) {
    if (vec) {
        if constexpr (sizeof(T) == 4) {
            const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
            const float4 a = p[0], b = p[1];
            f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
            f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
        } else {
            unpack8<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(base) + at), f);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = i < n ? to_f32(static_cast<const T*>(base)[at + i]) : 0.f;
    }
}

template <typename T>
__device__ __forceinline__ void store8(void* base, int64_t at, bool vec, int n, const float (&f)[8]) {
    if (vec) {
        if constexpr (sizeof(T) == 4) {
            float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
            p[0] = make_float4(f[0], f[1], f[2], f[3]);
            p[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            *reinterpret_cast<uint4*>(static_cast<T*>(base) + at) = pack8<T>(f);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) static_cast<T*>(base)[at + i] = from_f32<T>(f[i]);
    }
}

// Sixteen bytes at a row's byte `at`, whose address is a multiple of 16; those
// outside of the row's `bytes` read as zero and are not touched.
using Window = uint4;

__device__ __forceinline__ Window load_window(const uint8_t* row, int64_t at, int64_t bytes) {
    if (at >= 0 && at + 16 <= bytes) return *reinterpret_cast<const uint4*>(row + at);
    uint32_t w[4] = {};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (at + i >= 0 && at + i < bytes) w[i / 4] |= uint32_t(row[at + i]) << (8 * (i % 4));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ Window shuffle_window(const Window& w, int lane) {
    return make_uint4(__shfl_sync(0xffffffffu, w.x, lane), __shfl_sync(0xffffffffu, w.y, lane),
                      __shfl_sync(0xffffffffu, w.z, lane), __shfl_sync(0xffffffffu, w.w, lane));
}

// The 16 bytes from byte `off` on of two neighbouring windows.
__device__ __forceinline__ uint4 join_windows(const Window& a, const Window& b, int off) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (off & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (off & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const uint32_t bits = 8u * (uint32_t(off) & 3u);
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                      __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

}  // namespace tpg
