// Activations of the fused epilogues and their derivatives, in fp32.
//
// Every form is written so that fp32 keeps its relative accuracy in the tails and no finite input
// gives NaN: gelu through the normal distribution function (0.5 x (1 + erf) cancels for x < 0), the
// tanh form of gelu as x * sigmoid(2 y), sigmoid as 1 / (1 + exp(-x)) with exp overflowing to
// infinity (the quotient is then 0).  NaN inputs give NaN.
//
// The normal distribution function's tail is Phi(-|x|) = Q(t) exp(-x^2 / 2), t = 1 / (1 + P |x|), Q a
// polynomial fitted here (iteratively reweighted least squares of the relative error on |x| <= 14:
// at most 6.4e-7): two special-function instructions and ten multiply-adds, where the CUDA library's
// normcdff made the epilogue of a 128 x 160 tile take as long as its 32 groups' products.  The
// derivative needs the same exponential.
#pragma once

#include "common.cuh"

namespace w4 {

constexpr float kGeluA = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// 1 / (1 + exp(-x)): exact to a few fp32 ulps (far below the fp16 rounding that follows).  The
// denominator is in [1, inf]; above 2^126 the fast division gives 0, the limit.
__device__ __forceinline__ float sigmoid_f32(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

// Phi(x), and exp(-x^2 / 2).
__device__ __forceinline__ float normal_cdf(float x, float& density) {
    const float a = fabsf(x);
    density = __expf(-0.5f * a * a);
    const float t = __fdividef(1.0f, fmaf(0.265f, a, 1.0f));
    float q = fmaf(t, -0.0677901953458786f, 0.19528397917747498f);
    q = fmaf(t, q, -0.0663776695728302f);
    q = fmaf(t, q, 0.1425032913684845f);
    q = fmaf(t, q, 0.08294312655925751f);
    q = fmaf(t, q, 0.10783734917640686f);
    q = fmaf(t, q, 0.10559980571269989f);
    q *= t * density;
    return x < 0.0f ? q : 1.0f - q;
}

template <int ACT>
__device__ __forceinline__ float act_fwd(float x) {
    if constexpr (ACT == W4_ACT_RELU) return x < 0.0f ? 0.0f : x;
    if constexpr (ACT == W4_ACT_GELU) {
        float density;
        return x * normal_cdf(x, density);
    }
    if constexpr (ACT == W4_ACT_GELU_TANH) return x * sigmoid_f32(2.0f * kGeluA * fmaf(kGeluB * x * x, x, x));
    if constexpr (ACT == W4_ACT_SILU) return x * sigmoid_f32(x);
    return x;
}

// act'(x), and act(x) where the caller wants both (one exponential for the two).
template <int ACT>
__device__ __forceinline__ float act_grad(float x, float& fwd) {
    if constexpr (ACT == W4_ACT_RELU) {
        fwd = x < 0.0f ? 0.0f : x;
        return x > 0.0f ? 1.0f : (x <= 0.0f ? 0.0f : x);
    }
    if constexpr (ACT == W4_ACT_GELU) {
        // past |x| = 15 the density is 0 and Phi 0 or 1 in fp32; the clamp keeps inf * 0 out
        const float c = x > 15.0f ? 15.0f : (x < -15.0f ? -15.0f : x);
        float density;
        const float cdf = normal_cdf(c, density);
        fwd = x * cdf;
        return fmaf(c * 0.3989422804014327f, density, cdf);
    }
    if constexpr (ACT == W4_ACT_GELU_TANH) {
        // past |x| = 15 the sigmoid is 0 or 1 to the last bit and s (1 - s) is 0
        const float c = x > 15.0f ? 15.0f : (x < -15.0f ? -15.0f : x);
        const float x2 = c * c;
        const float s = sigmoid_f32(2.0f * kGeluA * fmaf(kGeluB * x2, c, c));
        fwd = x * s;
        return fmaf(c * s * (1.0f - s), 2.0f * kGeluA * fmaf(3.0f * kGeluB, x2, 1.0f), s);
    }
    if constexpr (ACT == W4_ACT_SILU) {
        const float c = x > 100.0f ? 100.0f : (x < -100.0f ? -100.0f : x);  // keeps inf * 0 out
        const float s = sigmoid_f32(c);
        fwd = x * s;
        return s * fmaf(c, 1.0f - s, 1.0f);
    }
    fwd = x;
    return x == x ? 1.0f : x;
}

}  // namespace w4
