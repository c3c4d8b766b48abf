// Activations of the operators and their derivatives, in fp32.
//
//   relu       max(z, 0)                                  z > 0
//   gelu       z Phi(z), Phi(z) = (1 + erf(z / sqrt 2)) / 2
//                                                         Phi(z) + z phi(z)
//   gelu_tanh  z (1 + t) / 2, t = tanh(c (z + a z^3)), c = sqrt(2 / pi),
//              a = 0.044715                (1 + t) / 2 + z (1 - t^2) c (1 + 3 a z^2) / 2
//   silu       z s(z), s(z) = 1 / (1 + exp(-z))           s (1 + z (1 - s))
//
// Phi by the rational approximation of erf in Abramowitz and Stegun, Handbook
// of Mathematical Functions, 7.1.26 (|error| <= 1.5e-7): with x = |z| / sqrt 2
// and t = 1 / (1 + p x), Phi(-|z|) = (a1 t + ... + a5 t^5) exp(-x^2) / 2, so the
// far negative side needs no cancelling difference and phi shares the
// exponential.  erff took the epilogue of a 256 x 256 tile from 3 to 5 us
// longer than none; this form costs what gelu_tanh does.
// tanh is taken as 2 s(2y) - 1 and s by one exponential and one fast divide
// (a few units in the last place of fp32; the results are rounded to bf16).
// Large arguments: exp overflows to infinity and s to 0, whose limits are the
// activations' own.
#pragma once

#include <type_traits>

#include "pgemm.h"

namespace pg {

__device__ __forceinline__ float sigmoid_f32(float z) {
    return __fdividef(1.0f, 1.0f + __expf(-z));
}

// Phi(z) and exp(-z^2 / 2)
__device__ __forceinline__ float normal_cdf(float z, float &e) {
    const float x = fabsf(z) * 0.70710678118654752f;
    const float t = __fdividef(1.0f, fmaf(0.3275911f, x, 1.0f));
    e = __expf(-0.5f * z * z);
    float p = fmaf(1.061405429f, t, -1.453152027f);
    p = fmaf(p, t, 1.421413741f);
    p = fmaf(p, t, -0.284496736f);
    p = fmaf(p, t, 0.254829592f);
    const float h = 0.5f * p * t * e;
    return z < 0.0f ? h : 1.0f - h;
}

// A fast divide returns 0 for divisors beyond 2^126, and exp(-z) of a large
// negative z is infinite: 1 / inf = 0 either way, so s(z) -> 0.
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == PGEMM_ACT_RELU) {
        return z < 0.0f ? 0.0f : z;  // a NaN stays one
    } else if constexpr (ACT == PGEMM_ACT_GELU) {
        float e;
        return z * normal_cdf(z, e);
    } else if constexpr (ACT == PGEMM_ACT_GELU_TANH) {
        const float y = 0.79788456080286536f * (z + 0.044715f * z * z * z);
        return z * sigmoid_f32(2.0f * y);
    } else if constexpr (ACT == PGEMM_ACT_SILU) {
        return z * sigmoid_f32(z);
    } else {
        return z;
    }
}

// value <- act(z), returns act'(z)
template <int ACT>
__device__ __forceinline__ float act_value_grad(float z, float &value) {
    if constexpr (ACT == PGEMM_ACT_RELU) {
        value = z < 0.0f ? 0.0f : z;
        return z > 0.0f ? 1.0f : 0.0f;
    } else if constexpr (ACT == PGEMM_ACT_GELU) {
        float e;
        const float cdf = normal_cdf(z, e);
        value = z * cdf;
        return fmaf(z * 0.39894228040143268f, e, cdf);
    } else if constexpr (ACT == PGEMM_ACT_GELU_TANH) {
        const float z2 = z * z;
        const float y = 0.79788456080286536f * z * (1.0f + 0.044715f * z2);
        const float s = sigmoid_f32(2.0f * y);  // (1 + t) / 2; (1 - t^2) / 2 = 2 s (1 - s)
        value = z * s;
        const float dy = 0.79788456080286536f * (1.0f + 0.134145f * z2);
        // far out s (1 - s) is 0 before dy overflows; keep 0 * inf away
        const float w = s * (1.0f - s);
        return w == 0.0f ? s : fmaf(2.0f * z * w, dy, s);
    } else if constexpr (ACT == PGEMM_ACT_SILU) {
        const float s = sigmoid_f32(z);
        value = z * s;
        return s * fmaf(z, 1.0f - s, 1.0f);
    } else {
        value = z;
        return 1.0f;
    }
}

// f(std::integral_constant<int, ACT>) for the runtime activation `act`: one
// uniform branch around the loops that use it.
template <class F>
__device__ __forceinline__ void with_act(int act, F &&f) {
    switch (act) {
        case PGEMM_ACT_RELU: f(std::integral_constant<int, PGEMM_ACT_RELU>{}); break;
        case PGEMM_ACT_GELU: f(std::integral_constant<int, PGEMM_ACT_GELU>{}); break;
        case PGEMM_ACT_GELU_TANH: f(std::integral_constant<int, PGEMM_ACT_GELU_TANH>{}); break;
        case PGEMM_ACT_SILU: f(std::integral_constant<int, PGEMM_ACT_SILU>{}); break;
        default: f(std::integral_constant<int, PGEMM_ACT_NONE>{}); break;
    }
}

}  // namespace pg
