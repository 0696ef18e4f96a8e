// Activations of the linear layer's epilogues (include/linear_epilogue.h) and their
// derivatives, in fp32.
//
// GELU's tanh form is x * sigma(2u) with u = sqrt(2/pi) (x + 0.044715 x^3) and sigma the
// logistic function, since (1 + tanh u) / 2 = sigma(2u): no cancellation for negative x,
// where 1 + tanh u has lost its digits. Its derivative is sigma + x sigma (1 - sigma) 2u',
// SiLU's sigma (1 + x (1 - sigma)), with 1 - sigma = e^-v sigma(v), which does not cancel
// either. The derivatives take |x| beyond a bound where sigma is 0 or 1 in fp32 as the
// bound, so that no infinity meets a zero.
//
// FAST (outputs of 8 significant bits): __expf and __fdividef, each off by a few 2^-23
// of its result over the arguments at hand; otherwise expf and an IEEE division.
#pragma once

#include "../../include/linear_epilogue.h"

#include <cuda_bf16.h>

#include <cstdint>

namespace mmbwd {
namespace act {

template <bool FAST>
__device__ __forceinline__ float exp_neg(float v) {
    return FAST ? __expf(-v) : expf(-v);
}
template <bool FAST>
__device__ __forceinline__ float quotient(float a, float b) {
    return FAST ? __fdividef(a, b) : a / b;
}

constexpr float GELU_K = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float GELU_C = 0.044715f;

template <int ACT, bool FAST>
__device__ __forceinline__ float value(float x) {
    if constexpr (ACT == MMBWD_ACT_GELU) {
        const float v = x * fmaf(2.f * GELU_K * GELU_C, x * x, 2.f * GELU_K);
        // (__fdividef gives a NaN for an infinite x over an infinite denominator and 0 for a
        // finite one over more than 2^126, where the quotient is 0 too)
        return quotient<FAST>(x, 1.f + exp_neg<FAST>(v));
    } else if constexpr (ACT == MMBWD_ACT_SILU) {
        return quotient<FAST>(x, 1.f + exp_neg<FAST>(x));
    } else if constexpr (ACT == MMBWD_ACT_RELU) {
        return x < 0.f ? 0.f : x;  // (a NaN is not below 0)
    } else {
        return x;
    }
}

// x between -b and b; a NaN stays one
__device__ __forceinline__ float within(float x, float b) { return x > b ? b : x < -b ? -b : x; }

template <int ACT, bool FAST>
__device__ __forceinline__ float slope(float x) {
    if constexpr (ACT == MMBWD_ACT_GELU) {
        x = within(x, 10.f);  // sigma(2u) is below 2^-125 at -10
        const float q = x * x;
        const float v = x * fmaf(2.f * GELU_K * GELU_C, q, 2.f * GELU_K);
        const float e = exp_neg<FAST>(v), s = quotient<FAST>(1.f, 1.f + e);
        const float rest = x * s * fmaf(6.f * GELU_K * GELU_C, q, 2.f * GELU_K);  // x sigma 2u'
        return fmaf(rest, e * s, s);
    } else if constexpr (ACT == MMBWD_ACT_SILU) {
        x = within(x, 87.f);  // e^87 is finite, sigma(-87) below 2^-125
        const float e = exp_neg<FAST>(x), s = quotient<FAST>(1.f, 1.f + e);
        return s * fmaf(x, e * s, 1.f);
    } else if constexpr (ACT == MMBWD_ACT_RELU) {
        return x > 0.f ? 1.f : x == x ? 0.f : x;  // (a NaN stays one)
    } else {
        return 1.f;
    }
}

// f(Act<ACT>) for the runtime `act`: the branch is taken once, outside the loops over values.
template <int ACT>
struct Act {
    static constexpr int value = ACT;
};
template <typename F>
__device__ __forceinline__ void with(int act, F f) {
    if (act == MMBWD_ACT_GELU) f(Act<MMBWD_ACT_GELU>{});
    else if (act == MMBWD_ACT_SILU) f(Act<MMBWD_ACT_SILU>{});
    else if (act == MMBWD_ACT_RELU) f(Act<MMBWD_ACT_RELU>{});
    else f(Act<MMBWD_ACT_NONE>{});
}

}  // namespace act
}  // namespace mmbwd
