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

// Pairs of 32-bit values in one 64-bit register: one instruction multiplies or
// adds both, which halves what the activations cost an epilogue (they are bound
// by instruction issue).
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ void split(F2 p, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v));
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
// 2^x, 1 / x and |x| of both.
__device__ __forceinline__ float ex2_of(float x) {
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ F2 exp2_2(F2 p) {
    float a, b;
    split(p, a, b);
    return f2(ex2_of(a), ex2_of(b));
}
__device__ __forceinline__ F2 recip_2(F2 p) {
    float a, b;
    split(p, a, b);
    return f2(__fdividef(1.f, a), __fdividef(1.f, b));
}
// min(|x|, 64) of both.
__device__ __forceinline__ F2 abs64_2(F2 p) {
    float a, b;
    split(p, a, b);
    return f2(fminf(fabsf(a), 64.f), fminf(fabsf(b), 64.f));
}
__device__ __forceinline__ F2 neg_2(F2 p) { return F2{p.v ^ 0x8000000080000000ull}; }
// max(x, 0); a NaN stays one.
__device__ __forceinline__ float relu_of(float x) {
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ F2 relu_2(F2 p) {
    float a, b;
    split(p, a, b);
    return f2(relu_of(a), relu_of(b));
}

constexpr float kLog2e = 1.4426950408889634f;

// The normal distribution's tail past a, erfc(a / sqrt 2) / 2, as 2^P(a): log2 of
// the tail is smooth, and P is its degree-8 polynomial over [0, 5.5], fitted
// here by weighted least squares to the smallest largest error of a times the
// tail (4.7e-8, evaluated in 32 bits); past that it falls on to -infinity. One
// branch-free exponential: erff takes two paths that a warp has to go through
// both, and a rational form needs a reciprocal besides, at 8 cycles of the
// special-function unit for a warp (gelu at 32 columns: 1400 cycles so).
__device__ __forceinline__ F2 normal_tail(F2 a) {
    F2 p = fma(a, f2(-1.6899085e-06f), f2(2.5076528e-05f));
    p = fma(a, p, f2(-0.00011442498f));
    p = fma(a, p, f2(-0.00032345162f));
    p = fma(a, p, f2(0.007333563f));
    p = fma(a, p, f2(-0.052714363f));
    p = fma(a, p, f2(-0.45911536f));
    p = fma(a, p, f2(-1.1511233f));
    p = fma(a, p, f2(-0.99999887f));
    return exp2_2(p);
}

// act(z) of a pair. The exponentials and reciprocals are the hardware's
// (relative error near 2^-21, far below a 16-bit output's rounding and about 8
// ulp of a 32-bit one's; a quotient by 2^126 or more is 0).
template <int ACT>
__device__ __forceinline__ F2 act_fwd(F2 z) {
    if constexpr (ACT == TPGEMM_ACT_RELU) return relu_2(z);
    if constexpr (ACT == TPGEMM_ACT_SILU)
        return mul(z, recip_2(add(exp2_2(mul(z, f2(-kLog2e))), f2(1.f))));
    if constexpr (ACT == TPGEMM_ACT_GELU) {
        // z Phi(z) = max(z, 0) - |z| tail(|z|); the tail is 0 from 14 on
        const F2 a = abs64_2(z);
        return fma(neg_2(a), normal_tail(a), relu_2(z));
    }
    if constexpr (ACT == TPGEMM_ACT_GELU_TANH) {
        // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u)), u = sqrt(2/pi) (z + 0.044715 z^3)
        const F2 u = mul(z, fma(mul(z, z), f2(-kLog2e * 1.5957691216057308f * 0.044715f),
                                f2(-kLog2e * 1.5957691216057308f)));
        return mul(z, recip_2(add(exp2_2(u), f2(1.f))));
    }
    return z;
}

// act'(z) of a pair.
template <int ACT>
__device__ __forceinline__ F2 act_bwd(F2 z) {
    if constexpr (ACT == TPGEMM_ACT_RELU) {
        float a, b;
        split(z, a, b);
        return f2(a > 0.f ? 1.f : 0.f, b > 0.f ? 1.f : 0.f);
    }
    if constexpr (ACT == TPGEMM_ACT_SILU) {
        const F2 s = recip_2(add(exp2_2(mul(z, f2(-kLog2e))), f2(1.f)));
        return mul(s, fma(z, fma(neg_2(s), f2(1.f), f2(1.f)), f2(1.f)));
    }
    if constexpr (ACT == TPGEMM_ACT_GELU) {
        // Phi(z) + z phi(z), Phi(z) = tail or 1 - tail
        const F2 e = exp2_2(mul(mul(z, z), f2(-0.5f * kLog2e)));
        const F2 q = normal_tail(abs64_2(z));
        float qa, qb, a, b;
        split(q, qa, qb);
        split(z, a, b);
        const F2 phi = f2(a > 0.f ? 1.f - qa : qa, b > 0.f ? 1.f - qb : qb);
        return fma(mul(z, f2(0.3989422804014327f)), e, phi);
    }
    if constexpr (ACT == TPGEMM_ACT_GELU_TANH) {
        const F2 z2 = mul(z, z);
        const F2 u = mul(z, fma(z2, f2(-kLog2e * 1.5957691216057308f * 0.044715f),
                                f2(-kLog2e * 1.5957691216057308f)));
        const F2 s = recip_2(add(exp2_2(u), f2(1.f)));
        // d(z s)/dz with ds/dz = s (1 - s) d(2u)/dz
        const F2 d = fma(z2, f2(1.5957691216057308f * 0.134145f), f2(1.5957691216057308f));
        return fma(mul(mul(z, s), fma(neg_2(s), f2(1.f), f2(1.f))), d, s);
    }
    return f2(1.f);
}

template <int ACT>
__device__ __forceinline__ float act_fwd(float z) {
    float a, b;
    split(act_fwd<ACT>(f2(z)), a, b);
    return a;
}
template <int ACT>
__device__ __forceinline__ float act_bwd(float z) {
    float a, b;
    split(act_bwd<ACT>(f2(z)), a, b);
    return a;
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
