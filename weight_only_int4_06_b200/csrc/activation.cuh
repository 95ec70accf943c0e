// Activations of the fused epilogues and their derivatives, in fp32, two elements at a time.
//
// An epilogue's arithmetic runs while the tensor cores wait for it, so its instruction count counts: the
// multiply-adds are packed (two fp32 in one instruction), the exponential is 2^(x log2 e) and the
// division a reciprocal, one special-function instruction each (2 ulp, far below the fp16 rounding that
// follows).  Every form keeps its relative accuracy in the tails and gives no NaN for finite inputs: gelu
// through the normal distribution function (0.5 x (1 + erf) cancels for x < 0), the tanh form of gelu as
// x * sigmoid(2 y), sigmoid as 1 / (1 + exp(-x)) with exp overflowing to infinity (the quotient is then
// 0).  NaN inputs give NaN, but for the identity's derivative: it is 1 everywhere.
//
// The normal distribution function's tail is Phi(-|x|) = Q(t) exp(-x^2 / 2), t = 1 / (1 + P |x|), Q a
// polynomial fitted here (iteratively reweighted least squares of the relative error on |x| <= 14:
// at most 7.2e-7); the derivative needs the same exponential.
#pragma once

#include "common.cuh"

namespace w4 {

// ------------------------------------------------------------------ two packed fp32
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ void split(F2 x, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v));
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
// Applied to each half.
template <typename F>
__device__ __forceinline__ F2 each(F2 x, F&& f) {
    float a, b;
    split(x, a, b);
    return f2(f(a), f(b));
}
__device__ __forceinline__ F2 exp2_2(F2 x) {
    return each(x, [](float a) {
        float r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
        return r;
    });
}
__device__ __forceinline__ F2 rcp_2(F2 x) {
    return each(x, [](float a) {
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
        return r;
    });
}
__device__ __forceinline__ F2 clamp_2(F2 x, float m) {  // NaN stays NaN
    return each(x, [m](float a) { return a > m ? m : (a < -m ? -m : a); });
}

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kGeluA = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;
constexpr float kRsqrt2Pi = 0.3989422804014327f;

// 1 / (1 + exp(-c x)).
__device__ __forceinline__ F2 sigmoid_2(F2 x, float c = 1.0f) {
    return rcp_2(add2(exp2_2(mul2(x, f2(-c * kLog2E))), f2(1.0f)));
}

// Phi(x), and exp(-x^2 / 2).
__device__ __forceinline__ F2 normal_cdf_2(F2 x, F2& density) {
    density = exp2_2(mul2(mul2(x, x), f2(-0.5f * kLog2E)));
    const F2 t = rcp_2(fma2(each(x, [](float a) { return fabsf(a); }), f2(0.265f), f2(1.0f)));
    F2 q = fma2(t, f2(-0.0677901953458786f), f2(0.19528397917747498f));
    q = fma2(t, q, f2(-0.0663776695728302f));
    q = fma2(t, q, f2(0.1425032913684845f));
    q = fma2(t, q, f2(0.08294312655925751f));
    q = fma2(t, q, f2(0.10783734917640686f));
    q = fma2(t, q, f2(0.10559980571269989f));
    q = mul2(mul2(q, t), density);
    float xa, xb, qa, qb;
    split(x, xa, xb);
    split(q, qa, qb);
    return f2(xa < 0.0f ? qa : 1.0f - qa, xb < 0.0f ? qb : 1.0f - qb);
}

template <int ACT>
__device__ __forceinline__ F2 act_fwd2(F2 x) {
    if constexpr (ACT == W4_ACT_RELU) return each(x, [](float a) { return a < 0.0f ? 0.0f : a; });
    if constexpr (ACT == W4_ACT_GELU) {
        F2 density;
        return mul2(x, normal_cdf_2(x, density));
    }
    if constexpr (ACT == W4_ACT_GELU_TANH)
        return mul2(x, sigmoid_2(fma2(mul2(mul2(x, f2(kGeluB)), x), x, x), 2.0f * kGeluA));
    if constexpr (ACT == W4_ACT_SILU) return mul2(x, sigmoid_2(x));
    return x;
}

// act'(x), and act(x) where the caller wants both (one exponential for the two).
template <int ACT>
__device__ __forceinline__ F2 act_grad2(F2 x, F2& fwd) {
    if constexpr (ACT == W4_ACT_RELU) {
        fwd = act_fwd2<ACT>(x);
        return each(x, [](float a) { return a > 0.0f ? 1.0f : (a <= 0.0f ? 0.0f : a); });
    }
    if constexpr (ACT == W4_ACT_GELU) {
        // past |x| = 15 the density is 0 and Phi 0 or 1 in fp32; the clamp keeps inf * 0 out
        const F2 c = clamp_2(x, 15.0f);
        F2 density;
        const F2 cdf = normal_cdf_2(c, density);
        fwd = mul2(x, cdf);
        return fma2(mul2(c, f2(kRsqrt2Pi)), density, cdf);
    }
    if constexpr (ACT == W4_ACT_GELU_TANH) {
        // past |x| = 15 the sigmoid is 0 or 1 to the last bit and s (1 - s) is 0
        const F2 c = clamp_2(x, 15.0f);
        const F2 b = mul2(mul2(c, c), f2(kGeluB));
        const F2 s = sigmoid_2(fma2(b, c, c), 2.0f * kGeluA);
        fwd = mul2(x, s);
        const F2 r = fma2(s, f2(-1.0f), f2(1.0f));
        return fma2(mul2(mul2(c, s), r), fma2(b, f2(6.0f * kGeluA), f2(2.0f * kGeluA)), s);
    }
    if constexpr (ACT == W4_ACT_SILU) {
        const F2 c = clamp_2(x, 100.0f);  // keeps inf * 0 out
        const F2 s = sigmoid_2(c);
        fwd = mul2(x, s);
        return mul2(s, fma2(c, fma2(s, f2(-1.0f), f2(1.0f)), f2(1.0f)));
    }
    fwd = x;
    return f2(1.0f);
}

template <int ACT>
__device__ __forceinline__ float act_fwd(float x) {
    float a, b;
    split(act_fwd2<ACT>(f2(x)), a, b);
    return a;
}

}  // namespace w4
