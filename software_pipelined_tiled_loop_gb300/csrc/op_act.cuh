// Activations of the operators and their derivatives, in fp32.
//
//   relu       max(z, 0)                                  z > 0
//   gelu       z Phi(z), Phi(z) = (1 + erf(z / sqrt 2)) / 2
//                                                         Phi(z) + z phi(z)
//   gelu_tanh  z (1 + t) / 2, t = tanh(c (z + a z^3)), c = sqrt(2 / pi),
//              a = 0.044715                (1 + t) / 2 + z (1 - t^2) c (1 + 3 a z^2) / 2
//   silu       z s(z), s(z) = 1 / (1 + exp(-z))           s (1 + z (1 - s))
//
// Phi(-|z|) = (a1 t + ... + a6 t^6) exp(-z^2 / 2), t = 1 / (1 + p |z|): the form of
// Abramowitz and Stegun's 7.1.26 with a term more and coefficients of its own, fitted by
// linear programming to exp(z^2 / 2) Phi(-|z|) on [0, 13.3] for the least largest relative
// error, weighted by 1 / (1 + 10 max(0, |z| - 1)).  Phi is within 3e-7 absolutely, and
// of the tail itself 7e-7 up to |z| = 1, 1.4e-5 up to 6 and 4.4e-5 up to 13, where it
// passes below 2^-126: gelu is good to bf16 on the far negative side too (7.1.26 itself,
// made for 1.5e-7 of erf, is off by 4e-3 of gelu at -6 and 1e-2 at -8).  phi shares the
// exponential.
// tanh is taken as 2 s(2y) - 1 and s by one ex2.approx and one rcp.approx (a few
// units in the last place of fp32; the results are rounded to bf16).  Large
// arguments: the exponential overflows to infinity and s to 0, whose limits are
// the activations' own.  What bounds an epilogue with an activation is the issue
// of these instructions (two warps a scheduler, 128 columns a lane), so each is
// spelled out with as few as it takes.
#pragma once

#include <type_traits>

#include "pgemm.h"

namespace pg {

// 2^x and 1 / x by the special-function unit, subnormals flushed to zero.
__device__ __forceinline__ float ex2_ftz(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_ftz(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// s(x) of the argument scaled by -log2(e): 2^(-x log2 e) overflows to infinity
// for large negative x, whose reciprocal is 0.
__device__ __forceinline__ float sigmoid_neg2(float x) { return rcp_ftz(1.0f + ex2_ftz(x)); }

// Phi(-|z|) and e = exp(-z^2 / 2)
__device__ __forceinline__ float normal_tail(float z, float &e) {
    const float t = rcp_ftz(fmaf(fabsf(z), 0.295f, 1.0f));
    e = ex2_ftz(z * z * -0.72134752044448170f);  // log2(e) / 2
    float p = fmaf(-0.0846582426f, t, 0.254261525f);
    p = fmaf(p, t, -0.0582768052f);
    p = fmaf(p, t, 0.163223048f);
    p = fmaf(p, t, 0.106952257f);
    p = fmaf(p, t, 0.118498125f);
    return p * t * e;
}

// c (z + a z^3) times -2 log2(e), the argument of sigmoid_neg2 for gelu_tanh:
// (1 + tanh y) / 2 = s(2 y)
constexpr float kTanhC = -2.0f * 0.79788456080286536f * 1.4426950408889634f;

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
    if constexpr (ACT == PGEMM_ACT_RELU) {
        return z < 0.0f ? 0.0f : z;  // a NaN stays one
    } else if constexpr (ACT == PGEMM_ACT_GELU) {
        float e;
        const float h = normal_tail(z, e);
        return z * (z < 0.0f ? h : 1.0f - h);
    } else if constexpr (ACT == PGEMM_ACT_GELU_TANH) {
        return z * sigmoid_neg2(z * fmaf(z * z, kTanhC * 0.044715f, kTanhC));
    } else if constexpr (ACT == PGEMM_ACT_SILU) {
        return z * sigmoid_neg2(z * -1.4426950408889634f);
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
        const float h = normal_tail(z, e);
        const float phi = z < 0.0f ? h : 1.0f - h;
        value = z * phi;
        return fmaf(z * 0.39894228040143268f, e, phi);
    } else if constexpr (ACT == PGEMM_ACT_GELU_TANH) {
        const float z2 = z * z;
        const float s = sigmoid_neg2(z * fmaf(z2, kTanhC * 0.044715f, kTanhC));
        value = z * s;
        // s + z (1 - t^2) y' / 2 with (1 - t^2) / 2 = 2 s (1 - s)
        const float dy = fmaf(z2, 2.0f * 0.79788456080286536f * 0.134145f,
                              2.0f * 0.79788456080286536f);
        // far out s (1 - s) is 0 before dy overflows; keep 0 * inf away
        const float w = s * (1.0f - s);
        return w == 0.0f ? s : fmaf(z * w, dy, s);
    } else if constexpr (ACT == PGEMM_ACT_SILU) {
        const float s = sigmoid_neg2(z * -1.4426950408889634f);
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
