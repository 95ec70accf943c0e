// Activations of the fused epilogues and their derivatives, in fp32.
//
// Every form is written so that fp32 keeps its relative accuracy in the tails and no finite input
// gives NaN: gelu through the normal distribution function (0.5 x (1 + erf) cancels for x < 0), the
// tanh form of gelu as x * sigmoid(2 y), sigmoid as 1 / (1 + exp(-x)) with exp overflowing to
// infinity (the quotient is then 0).  NaN inputs give NaN.
#pragma once

#include "common.cuh"

namespace w4 {

constexpr float kGeluA = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// 1 / (1 + exp(-x)): exact to a few fp32 ulps (far below the fp16 rounding that follows).  The
// denominator is in [1, inf]; above 2^126 the fast division gives 0, the limit.
__device__ __forceinline__ float sigmoid_f32(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

template <int ACT>
__device__ __forceinline__ float act_fwd(float x) {
    if constexpr (ACT == W4_ACT_RELU) return x < 0.0f ? 0.0f : x;
    if constexpr (ACT == W4_ACT_GELU) return x * normcdff(x);
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
        const float cdf = normcdff(x);
        // x * exp(-x^2/2): past |x| = 15 the product is 0 in fp32; the clamp keeps inf * 0 out
        const float c = x > 15.0f ? 15.0f : (x < -15.0f ? -15.0f : x);
        fwd = x * cdf;
        return fmaf(c * 0.3989422804014327f, __expf(-0.5f * c * c), cdf);
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
