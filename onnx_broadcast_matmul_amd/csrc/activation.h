// activation.h -- the gated block's activations f and their derivatives, in
// FP32.  Each is written so that neither tail cancels: the sigmoid and its
// complement come from one exponential of -|x|, gelu from erfc, and the tanh
// form of gelu from (1 + tanh z) / 2 = sigmoid(2 z).
#pragma once

#include <hip/hip_runtime.h>

#include "mm.h"

namespace mm {

// sigmoid(x) and 1 - sigmoid(x).  EXACT (FP32 operands): the library
// exponential and a rounded division; otherwise the hardware's exponential and
// reciprocal, off by a few 2^-22, far below a 16-bit result's half step.
template <bool EXACT>
__device__ __forceinline__ void sigmoid_pair(float x, float &s, float &c) {
    const float e = EXACT ? expf(-fabsf(x)) : __expf(-fabsf(x));
    const float d = 1.0f + e;
    const float hi = EXACT ? 1.0f / d : __builtin_amdgcn_rcpf(d);
    const float lo = e * hi;
    s = x >= 0.0f ? hi : lo;
    c = x >= 0.0f ? lo : hi;
    if (x != x) s = c = x;
}

constexpr float kGeluC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

template <int ACT, bool EXACT>
__device__ __forceinline__ float act_value(float g) {
    float s, c;
    if constexpr (ACT == MM_ACT_RELU) {
        return g > 0.0f || g != g ? g : 0.0f;
    } else if constexpr (ACT == MM_ACT_GELU) {
        return g * (0.5f * erfcf(g * -0.70710678118654752f));
    } else if constexpr (ACT == MM_ACT_GELU_TANH) {
        sigmoid_pair<EXACT>(kGeluC * (g + kGeluA * g * g * g), s, c);
        return g * s;
    } else {
        sigmoid_pair<EXACT>(g, s, c);
        return ACT == MM_ACT_SILU ? g * s : s;
    }
}

// f(g) and f'(g).
template <int ACT, bool EXACT>
__device__ __forceinline__ void act_grad(float g, float &f, float &d) {
    float s, c;
    if constexpr (ACT == MM_ACT_RELU) {
        const bool on = g > 0.0f;
        f = on || g != g ? g : 0.0f;
        d = on ? 1.0f : 0.0f;
    } else if constexpr (ACT == MM_ACT_GELU) {
        const float p = 0.5f * erfcf(g * -0.70710678118654752f);
        const float q = EXACT ? expf(-0.5f * g * g) : __expf(-0.5f * g * g);
        f = g * p;
        d = p + g * q * 0.3989422804014327f;
    } else if constexpr (ACT == MM_ACT_GELU_TANH) {
        sigmoid_pair<EXACT>(kGeluC * (g + kGeluA * g * g * g), s, c);
        f = g * s;
        d = s + g * s * c * kGeluC * (1.0f + 3.0f * kGeluA * g * g);
    } else {
        sigmoid_pair<EXACT>(g, s, c);
        if constexpr (ACT == MM_ACT_SILU) {
            f = g * s;
            d = s * (1.0f + g * c);
        } else {
            f = s;
            d = s * c;
        }
    }
}

// INT8 product's epilogue: the exact integer sum, rounded to FP32 once (the
// sum can need 31 bits), times the scales, plus the bias.
__device__ __forceinline__ float scaled_value(int acc, float sa, float sb, float bias) {
    return (float)acc * sa * sb + bias;
}

}  // namespace mm
