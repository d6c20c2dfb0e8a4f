// Element types of the operators around the multiply, and the linear layer's
// epilogue for one output.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ops_internal.h"

namespace tpg {

using e4m3 = __nv_fp8_e4m3;
using e5m2 = __nv_fp8_e5m2;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(e4m3 v) { return float(v); }
__device__ __forceinline__ float to_f32(e5m2 v) { return float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v) {
    if constexpr (sizeof(T) == 4)
        return v;
    else if constexpr (std::is_same<T, __half>::value)
        return __float2half_rn(v);
    else if constexpr (std::is_same<T, __nv_bfloat16>::value)
        return __float2bfloat16_rn(v);
    else
        return T(v);  // 8 bits: round to nearest even, saturating
}

// The normal distribution's tail past |z|, given e = exp(-z^2 / 2): erfc(|z| /
// sqrt 2) / 2 by the rational approximation 7.1.26 of Abramowitz and Stegun's
// Handbook of Mathematical Functions (absolute error of erf below 1.5e-7; and
// no cancellation for negative z). One branch-free evaluation for all lanes:
// erff takes two paths that a warp has to go through both.
__device__ __forceinline__ float normal_tail(float z, float e) {
    const float t = __fdividef(1.f, 1.f + 0.3275911f * 0.70710678118654752f * fabsf(z));
    const float s = t * (0.254829592f +
                         t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
    return 0.5f * s * e;
}

// act(z). The exponentials and divisions are the hardware's (relative error near
// 2^-21, far below a 16-bit output's rounding and about 8 ulp of a 32-bit
// one's; a quotient by 2^126 or more is 0).
template <int ACT>
__device__ __forceinline__ float act_fwd(float z) {
    if constexpr (ACT == TPGEMM_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
    if constexpr (ACT == TPGEMM_ACT_SILU) return __fdividef(z, 1.f + __expf(-z));
    if constexpr (ACT == TPGEMM_ACT_GELU) {
        const float q = normal_tail(z, __expf(-0.5f * z * z));
        return z * (z > 0.f ? 1.f - q : q);
    }
    if constexpr (ACT == TPGEMM_ACT_GELU_TANH) {
        // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u)), u = sqrt(2/pi) (z + 0.044715 z^3)
        const float u2 = 1.5957691216057308f * (z + 0.044715f * z * z * z);
        return __fdividef(z, 1.f + __expf(-u2));
    }
    return z;
}

// act'(z).
template <int ACT>
__device__ __forceinline__ float act_bwd(float z) {
    if constexpr (ACT == TPGEMM_ACT_RELU) return z > 0.f ? 1.f : 0.f;
    if constexpr (ACT == TPGEMM_ACT_SILU) {
        const float s = __fdividef(1.f, 1.f + __expf(-z));
        return s * (1.f + z * (1.f - s));
    }
    if constexpr (ACT == TPGEMM_ACT_GELU) {
        const float e = __expf(-0.5f * z * z);
        const float q = normal_tail(z, e);
        return (z > 0.f ? 1.f - q : q) + z * 0.3989422804014327f * e;
    }
    if constexpr (ACT == TPGEMM_ACT_GELU_TANH) {
        const float z2 = z * z;
        const float u2 = 1.5957691216057308f * (z + 0.044715f * z * z2);
        const float s = __fdividef(1.f, 1.f + __expf(-u2));
        // d(z s)/dz with ds/dz = s (1 - s) d(2u)/dz
        return s + z * s * (1.f - s) * 1.5957691216057308f * (1.f + 0.134145f * z2);
    }
    return 1.f;
}

// Calls f(integral_constant<act>) for a run-time activation.
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
    switch (act) {
        case TPGEMM_ACT_RELU: f(std::integral_constant<int, TPGEMM_ACT_RELU>()); break;
        case TPGEMM_ACT_SILU: f(std::integral_constant<int, TPGEMM_ACT_SILU>()); break;
        case TPGEMM_ACT_GELU: f(std::integral_constant<int, TPGEMM_ACT_GELU>()); break;
        case TPGEMM_ACT_GELU_TANH: f(std::integral_constant<int, TPGEMM_ACT_GELU_TANH>()); break;
        default: f(std::integral_constant<int, TPGEMM_ACT_NONE>()); break;
    }
}

// The epilogue of output (m, n), in 32 bits until the one rounding of each store.
template <typename T, int ACT>
__device__ __forceinline__ void epilogue_one(const Epilogue& e, int64_t m, int64_t n, float x) {
    if (e.sa) x *= e.sa[m];
    if (e.sw) x *= e.sw[n];
    if (e.bias) x += to_f32(static_cast<const T*>(e.bias)[n]);
    if (e.Z) static_cast<T*>(e.Z)[m * e.ldz + n] = from_f32<T>(x);
    x = act_fwd<ACT>(x);
    if (e.R) x += to_f32(static_cast<const T*>(e.R)[m * e.ldr + n]);
    static_cast<T*>(e.Y)[m * e.ldy + n] = from_f32<T>(x);
}

}  // namespace tpg
