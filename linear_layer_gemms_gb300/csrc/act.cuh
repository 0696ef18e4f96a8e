// Activations of the linear layer's epilogues (include/linear_epilogue.h) and their
// derivatives, in fp32.
//
// GELU's tanh form is x * sigma(2u) with u = sqrt(2/pi) (x + 0.044715 x^3) and sigma the
// logistic function, since (1 + tanh u) / 2 = sigma(2u): no cancellation for negative x,
// where 1 + tanh u has lost its digits. Its derivative is sigma (1 + x (1 - sigma) 2u'),
// SiLU's sigma (1 + x (1 - sigma)), with 1 - sigma = e^-v sigma(v), which does not cancel
// either. The derivatives take |x| beyond a bound where sigma is 0 or 1 in fp32 as the
// bound, so that no infinity meets a zero.
//
// FAST (bf16 outputs, and fp32 ones where the epilogue's instructions slow the tensor
// cores down): exponential and reciprocal from one instruction each (ex2.approx.ftz and
// rcp.approx.ftz, relative errors of some 2^-22 over all arguments), and two values to
// an instruction in between; otherwise expf and an IEEE division.
#pragma once

#include "../../include/linear_epilogue.h"

#include <cuda_bf16.h>

#include <cstdint>

namespace mmbwd {
namespace act {

constexpr float GELU_K = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float GELU_C = 0.044715f;
constexpr float LOG2E = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float reciprocal_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Two fp32 values, worked on by one instruction.
struct Two {
    unsigned long long v;
    __device__ static Two of(float a, float b) {
        Two r;
        asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
        return r;
    }
    __device__ static Two both(float a) { return of(a, a); }
    __device__ float lo() const { return __uint_as_float(static_cast<uint32_t>(v)); }
    __device__ float hi() const { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
};
__device__ __forceinline__ Two fma(Two a, Two b, Two c) {
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ Two add(Two a, Two b) {
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Two mul(Two a, Two b) {
    Two r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

// x between -b and b; a NaN stays one
__device__ __forceinline__ float within(float x, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(b));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(r), "f"(-b));
    return r;
}

// act(x)
template <int ACT>
__device__ __forceinline__ float value(float x) {
    if constexpr (ACT == MMBWD_ACT_GELU) {
        const float v = x * fmaf(2.f * GELU_K * GELU_C, x * x, 2.f * GELU_K);
        return x / (1.f + expf(-v));
    } else if constexpr (ACT == MMBWD_ACT_SILU) {
        return x / (1.f + expf(-x));
    } else if constexpr (ACT == MMBWD_ACT_RELU) {
        return x < 0.f ? 0.f : x;  // (a NaN is not below 0)
    } else {
        return x;
    }
}

// act'(x)
template <int ACT>
__device__ __forceinline__ float slope(float x) {
    if constexpr (ACT == MMBWD_ACT_GELU) {
        x = within(x, 10.f);  // sigma(2u) is below 2^-125 at -10
        const float q = x * x;
        const float e = expf(-x * fmaf(2.f * GELU_K * GELU_C, q, 2.f * GELU_K)), s = 1.f / (1.f + e);
        const float rest = x * s * fmaf(6.f * GELU_K * GELU_C, q, 2.f * GELU_K);  // x sigma 2u'
        return fmaf(rest, e * s, s);
    } else if constexpr (ACT == MMBWD_ACT_SILU) {
        x = within(x, 87.f);  // e^87 is finite, sigma(-87) below 2^-125
        const float e = expf(-x), s = 1.f / (1.f + e);
        return s * fmaf(x, e * s, 1.f);
    } else if constexpr (ACT == MMBWD_ACT_RELU) {
        return x > 0.f ? 1.f : x == x ? 0.f : x;  // (a NaN stays one)
    } else {
        return 1.f;
    }
}

// The logistic function 1 / (1 + e), e = 2^t.
__device__ __forceinline__ Two exponential(Two t) { return Two::of(exp2_fast(t.lo()), exp2_fast(t.hi())); }
__device__ __forceinline__ Two logistic(Two e) {
    const Two d = add(e, Two::both(1.f));
    return Two::of(reciprocal_fast(d.lo()), reciprocal_fast(d.hi()));
}

// FAST, on a pair of values in place.
template <int ACT>
__device__ __forceinline__ void value_fast(float& a, float& b) {
    if constexpr (ACT == MMBWD_ACT_GELU || ACT == MMBWD_ACT_SILU) {
        const Two x = Two::of(a, b);
        Two t;
        if constexpr (ACT == MMBWD_ACT_GELU)
            t = mul(x, fma(mul(x, x), Two::both(-2.f * GELU_K * GELU_C * LOG2E), Two::both(-2.f * GELU_K * LOG2E)));
        else
            t = mul(x, Two::both(-LOG2E));
        const Two y = mul(x, logistic(exponential(t)));
        a = y.lo(), b = y.hi();
    } else {
        a = value<ACT>(a), b = value<ACT>(b);
    }
}

// act' of the pair x, times the pair d, into d. 1 - sigma = e sigma here too: as a subtraction
// it would be off by 2^-25 where it is small, which the factor x 2u' makes 2e-6 of GELU's
// derivative near x = 5, ten times the error of `slope`.
template <int ACT>
__device__ __forceinline__ void slope_fast(float& d0, float& d1, float x0, float x1) {
    if constexpr (ACT == MMBWD_ACT_GELU || ACT == MMBWD_ACT_SILU) {
        constexpr float LIMIT = ACT == MMBWD_ACT_GELU ? 10.f : 87.f;
        const Two x = Two::of(within(x0, LIMIT), within(x1, LIMIT));
        Two t, dv;  // the exponent, v'
        if constexpr (ACT == MMBWD_ACT_GELU) {
            const Two q = mul(x, x);
            t = mul(x, fma(q, Two::both(-2.f * GELU_K * GELU_C * LOG2E), Two::both(-2.f * GELU_K * LOG2E)));
            dv = fma(q, Two::both(6.f * GELU_K * GELU_C), Two::both(2.f * GELU_K));
        } else {
            t = mul(x, Two::both(-LOG2E));
            dv = Two::both(1.f);
        }
        const Two e = exponential(t), s = logistic(e), rest = mul(e, s);
        const Two y = mul(mul(Two::of(d0, d1), s), fma(mul(x, dv), rest, Two::both(1.f)));
        d0 = y.lo(), d1 = y.hi();
    } else {
        d0 *= slope<ACT>(x0), d1 *= slope<ACT>(x1);
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
