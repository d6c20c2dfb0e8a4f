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
// max(-|x|, -16) and min(x, y) of both.
__device__ __forceinline__ F2 minus_abs16_2(F2 p) {
    float a, b;
    split(p, a, b);
    return f2(fmaxf(-fabsf(a), -16.f), fmaxf(-fabsf(b), -16.f));
}
__device__ __forceinline__ F2 min_2(F2 p, F2 q) {
    float a, b, c, d;
    split(p, a, b);
    split(q, c, d);
    return f2(fminf(a, c), fminf(b, d));
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

// The normal distribution's tail past a in [0, 16], erfc(a / sqrt 2) / 2, as
// 2^P(m), m = -a: log2 of the tail is smooth, and P is a polynomial over [-13.2,
// 0] (past which a times the tail leaves 32 bits' normal numbers), fitted here by
// weighted least squares to the smallest largest error of two kinds at once: of the tail, and of
// the tail relative to itself, so that a negative z's gelu, though small, keeps
// its size. Evaluated in 32 bits:
//   degree 8   off by 5.3e-7, by 1e-4 of itself up to a = 4, 1.4e-4 up to 4.4 (where
//              an f16 result ends), 1.2e-3 anywhere: under half of a 16-bit
//              result's own rounding;
//   FINE (12)  off by 5.5e-8, by 4.7e-6 of itself up to 3, 3.2e-5 up to 4, 3.5e-4
//              anywhere: for 32-bit results. Half as much work again (4096 x 4096
//              x 64 with gelu 25.7 us, 24.0 of degree 8).
// P(-16) is below -189, so the tail ends at 0. One branch-free exponential: erff
// takes two paths that a warp has to go through both, and a rational form needs a
// reciprocal besides, at 8 cycles of the special-function unit for a warp (gelu
// at 32 columns: 1400 cycles so).
template <bool FINE>
__device__ __forceinline__ F2 normal_tail(F2 m) {
    F2 p;
    if constexpr (FINE) {
        p = fma(m, f2(-1.77966791e-11f), f2(-1.30777622e-09f));
        p = fma(m, p, f2(-4.15794723e-08f));
        p = fma(m, p, f2(-7.47283934e-07f));
        p = fma(m, p, f2(-8.27881195e-06f));
        p = fma(m, p, f2(-5.6687426e-05f));
        p = fma(m, p, f2(-0.000204559736f));
        p = fma(m, p, f2(0.000161342788f));
        p = fma(m, p, f2(0.00714332843f));
        p = fma(m, p, f2(0.0525699668f));
        p = fma(m, p, f2(-0.459180653f));
        p = fma(m, p, f2(1.15110874f));
        p = fma(m, p, f2(-0.99999994f));
    } else {
        p = fma(m, f2(3.89714749e-08f), f2(2.379222e-06f));
        p = fma(m, p, f2(6.1675637e-05f));
        p = fma(m, p, f2(0.000899372157f));
        p = fma(m, p, f2(0.00833507441f));
        p = fma(m, p, f2(0.0536045954f));
        p = fma(m, p, f2(-0.458758682f));
        p = fma(m, p, f2(1.15117025f));
        p = fma(m, p, f2(-0.999998569f));
    }
    return exp2_2(p);
}

// act(z) of a pair, FINE for a 32-bit result. silu and gelu_tanh multiply z by
// 1 / (1 + 2^u) with the hardware's exponential and reciprocal: off by about 2^-21
// of themselves, and by |u| 2^-24 more where 2^u is large (u is rounded to 32
// bits); a quotient by 2^126 or more is 0. gelu: see normal_tail.
template <int ACT, bool FINE>
__device__ __forceinline__ F2 act_fwd(F2 z) {
    if constexpr (ACT == TPGEMM_ACT_RELU) return relu_2(z);
    if constexpr (ACT == TPGEMM_ACT_SILU)
        return mul(z, recip_2(add(exp2_2(mul(z, f2(-kLog2e))), f2(1.f))));
    if constexpr (ACT == TPGEMM_ACT_GELU) {
        // z Phi(z) = max(z, 0) - |z| tail(|z|). A large positive z is held to 16
        // there too, a negative one is not: -infinity meets a tail of 0, which is
        // the formula's NaN.
        const F2 m = minus_abs16_2(z);
        return fma(min_2(z, m), normal_tail<FINE>(m), relu_2(z));
    }
    if constexpr (ACT == TPGEMM_ACT_GELU_TANH) {
        // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u)), u = sqrt(2/pi) (z + 0.044715 z^3)
        const F2 u = mul(z, fma(mul(z, z), f2(-kLog2e * 1.5957691216057308f * 0.044715f),
                                f2(-kLog2e * 1.5957691216057308f)));
        return mul(z, recip_2(add(exp2_2(u), f2(1.f))));
    }
    return z;
}

// act'(z) of a pair, as exactly as a 16-bit dZ needs it.
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
        const F2 q = normal_tail<false>(minus_abs16_2(z));
        float qa, qb, a, b;
        split(q, qa, qb);
        split(z, a, b);
        const F2 phi = f2(a > 0.f ? 1.f - qa : qa, b > 0.f ? 1.f - qb : qb);
        return fma(mul(z, f2(0.3989422804014327f)), e, phi);
    }
    if constexpr (ACT == TPGEMM_ACT_GELU_TANH) {
        // (z^2 of finite z stays finite: s is 0 or 1 long before 2^40.)
        const F2 z2 = min_2(mul(z, z), f2(1.09951163e12f));
        const F2 u = mul(z, fma(z2, f2(-kLog2e * 1.5957691216057308f * 0.044715f),
                                f2(-kLog2e * 1.5957691216057308f)));
        const F2 s = recip_2(add(exp2_2(u), f2(1.f)));
        // d(z s)/dz with ds/dz = s (1 - s) d(2u)/dz
        const F2 d = fma(z2, f2(1.5957691216057308f * 0.134145f), f2(1.5957691216057308f));
        return fma(mul(mul(z, s), fma(neg_2(s), f2(1.f), f2(1.f))), d, s);
    }
    return f2(1.f);
}

template <int ACT, bool FINE>
__device__ __forceinline__ float act_fwd(float z) {
    float a, b;
    split(act_fwd<ACT, FINE>(f2(z)), a, b);
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
    x = act_fwd<ACT, sizeof(T) == 4>(x);
    if (e.R) x += to_f32(static_cast<const T*>(e.R)[m * e.ldr + n]);
    static_cast<T*>(e.Y)[m * e.ldy + n] = from_f32<T>(x);
}

}  // namespace tpg
