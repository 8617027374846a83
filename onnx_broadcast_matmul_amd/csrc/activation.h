// activation.h -- the feed-forward operators' activations f and their derivatives, in
// FP32.  Each is written so that neither tail cancels: the sigmoid and its
// complement come from one exponential of -|x|, the tanh form of gelu from
// (1 + tanh z) / 2 = sigmoid(2 z), and gelu from the normal distribution's
// tail, whose exponential is also the density that the derivative needs.
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

// Normal distribution at g: P = Phi(g) and its density D.  The tail is
//   1 - Phi(|g|) = exp(-g^2 / 2) e(|g| / sqrt 2) / 2,  e(z) = exp(z^2) erfc(z),
// and e is smooth in q = 1 / (1 + p z): e(z) = q (c0 + c1 q + ...), fitted here
// by least squares on Chebyshev points, reweighted towards the least largest
// relative error over 0 <= z <= 14 (past that the tail is below FP32):
// 2.7e-6 with 7 coefficients, a hundredth of an FP16 half step; EXACT: 1.0e-8
// with 10, and the rounding of g^2 is put back into the exponential.  (The
// library's erfc cost about as much as the matrix work of a 1024-long K.)
template <bool EXACT>
__device__ __forceinline__ void normal_pair(float g, float &P, float &D) {
    const float a = fminf(fabsf(g), 40.0f);
    const float z = a * 0.70710678118654752f;
    const float h = a * a;
    float e, x;
    if constexpr (EXACT) {
        const float q = 1.0f / (1.0f + 0.35f * z);
        e = 4.184608091e-02f;
        e = e * q - 1.779090892e-01f;
        e = e * q + 2.267881683e-01f;
        e = e * q - 8.915867565e-02f;
        e = e * q + 1.390371659e-01f;
        e = e * q + 1.175938350e-01f;
        e = e * q + 1.612167270e-01f;
        e = e * q + 1.857080195e-01f;
        e = e * q + 1.974081938e-01f;
        e = e * q + 1.974695846e-01f;
        e *= q;
        x = expf(-0.5f * h) * (1.0f - 0.5f * fmaf(a, a, -h));
    } else {
        const float q = __builtin_amdgcn_rcpf(1.0f + 0.5f * z);
        e = 8.212535751e-02f;
        e = e * q - 3.356935106e-01f;
        e = e * q + 3.603833506e-01f;
        e = e * q + 5.776401879e-02f;
        e = e * q + 2.743037532e-01f;
        e = e * q + 2.788714043e-01f;
        e = e * q + 2.822429085e-01f;
        e *= q;
        x = __expf(-0.5f * h);
    }
    const float tail = 0.5f * e * x;
    P = g >= 0.0f ? 1.0f - tail : tail;
    D = x * 0.3989422804014327f;
}

constexpr float kGeluC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

template <int ACT, bool EXACT>
__device__ __forceinline__ float act_value(float g) {
    float s, c;
    if constexpr (ACT == MM_ACT_RELU) {
        return g > 0.0f || g != g ? g : 0.0f;
    } else if constexpr (ACT == MM_ACT_GELU) {
        normal_pair<EXACT>(g, s, c);
        return g * s;
    } else if constexpr (ACT == MM_ACT_GELU_TANH) {
        sigmoid_pair<EXACT>(kGeluC * (g + kGeluA * g * g * g), s, c);
        return g * s;
    } else {
        sigmoid_pair<EXACT>(g, s, c);
        return ACT == MM_ACT_SILU ? g * s : s;
    }
}

// f(z) where its derivative is not wanted, for 16-bit results: sigmoid(x) = 1 /
// (1 + 2^(-x log2 e)) needs no other tail (2^(..) overflows to infinity, whose
// reciprocal is the 0 that belongs there) and takes half the pair's instructions
// (8192 x 4096 x 11008 BF16 with tanh gelu: 8 us more than without, so 29).
template <int ACT, bool EXACT>
__device__ __forceinline__ float act_only(float z) {
    constexpr float L = 1.4426950408889634f;  // log2 e
    if constexpr (EXACT || ACT == MM_ACT_RELU || ACT == MM_ACT_GELU) {
        return act_value<ACT, EXACT>(z);
    } else if constexpr (ACT == MM_ACT_GELU_TANH) {
        const float x = z * fmaf(z * z, -L * kGeluC * kGeluA, -L * kGeluC);
        return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x));
    } else {
        const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-L * z));
        return ACT == MM_ACT_SILU ? z * s : s;
    }
}

// The same for an activation known at run time (MM_ACT_NONE: z).
template <bool EXACT>
__device__ __forceinline__ float act_run(int act, float z) {
    switch (act) {
    case MM_ACT_SILU: return act_only<MM_ACT_SILU, EXACT>(z);
    case MM_ACT_GELU: return act_only<MM_ACT_GELU, EXACT>(z);
    case MM_ACT_GELU_TANH: return act_only<MM_ACT_GELU_TANH, EXACT>(z);
    case MM_ACT_RELU: return act_only<MM_ACT_RELU, EXACT>(z);
    case MM_ACT_SIGMOID: return act_only<MM_ACT_SIGMOID, EXACT>(z);
    }
    return z;
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
        normal_pair<EXACT>(g, s, c);
        f = g * s;
        d = s + g * c;
    } else if constexpr (ACT == MM_ACT_GELU_TANH) {
        sigmoid_pair<EXACT>(kGeluC * (g + kGeluA * g * g * g), s, c);
        f = g * s;
        // s c is 0 long before g^2 leaves FP32, which the limit keeps finite:
        // the far finite gates' second term is 0 and not 0 times infinity.
        d = s + g * s * c * kGeluC * (1.0f + 3.0f * kGeluA * fminf(g * g, 1e30f));
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

// INT8 product's epilogue: the exact integer sum, rounded to FP32 (it can need
// 31 bits), times the row's scale, rounded; that times the column's scale plus
// the bias, rounded once.  The operations are spelled out, and the FP32 result
// kept apart from the narrowing (which the compiler else merges into the last
// operation here and there, rounding once where other kernels round twice), so
// that every kernel gives the same bits.
__device__ __forceinline__ float scaled_value(int acc, float sa, float sb, float bias) {
    float y = fmaf((float)acc * sa, sb, bias);
    asm("" : "+v"(y));
    return y;
}

}  // namespace mm
