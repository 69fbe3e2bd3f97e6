// gate_act.cuh -- the gate's activations and their derivatives, in fp32.
//
// With s(v) = 1/(1 + exp(-v)):
//   silu       g s(g)                       s (1 + g (1 - s))
//   gelu       g P(g), P(g) = erfc(-g/sqrt 2)/2     P + g exp(-g^2/2)/sqrt(2 pi)
//   gelu_tanh  g s(2v), v = sqrt(2/pi)(g + 0.044715 g^3)   (the same as g(1 + tanh v)/2)
//                                           s + 2 g s (1 - s) dv/dg
//   relu       max(g, 0)                    g > 0
//   sigmoid    s(g)                         s (1 - s)
// The forms keep their relative precision for large negative g, where 1 + tanh and
// 1 + erf cancel.  exp and the quotient are the fast device functions: relative
// errors of a few 2^-23 (times |v| for the exponential), far below a 16-bit result's.
#pragma once

#include "common.cuh"

namespace dgrad {

enum GateAct : int { kSilu = 0, kGelu = 1, kGeluTanh = 2, kRelu = 3, kSigmoid = 4 };

__device__ __forceinline__ float logistic(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

constexpr float kTanhA = 0.7978845608028654f;             // sqrt(2/pi)
constexpr float kTanhB = 0.7978845608028654f * 0.044715f;

__device__ __forceinline__ float gate_act(int act, float g)
{
    switch (act) {
    case kSilu: return g * logistic(g);
    case kGelu: return g * (0.5f * erfcf(g * -0.7071067811865476f));
    case kGeluTanh: return g * logistic(2.0f * g * fmaf(kTanhB * g, g, kTanhA));
    case kRelu: return g <= 0.f ? 0.f : g;
    default: return logistic(g);
    }
}

// act(g) and act'(g).
__device__ __forceinline__ float2 gate_act_grad(int act, float g)
{
    switch (act) {
    case kSilu: {
        const float s = logistic(g);
        return make_float2(g * s, s * fmaf(g, 1.0f - s, 1.0f));
    }
    case kGelu: {
        const float p = 0.5f * erfcf(g * -0.7071067811865476f);
        return make_float2(g * p, fmaf(g * 0.3989422804014327f, __expf(-0.5f * g * g), p));
    }
    case kGeluTanh: {
        const float s = logistic(2.0f * g * fmaf(kTanhB * g, g, kTanhA));
        const float dv = fminf(fmaf(3.0f * kTanhB * g, g, kTanhA), 1e30f);   // finite: s (1 - s) is 0 there
        return make_float2(g * s, fmaf(2.0f * g * s * (1.0f - s), dv, s));
    }
    case kRelu: return make_float2(g <= 0.f ? 0.f : g, g > 0.f ? 1.0f : 0.f);
    default: {
        const float s = logistic(g);
        return make_float2(s, s * (1.0f - s));
    }
    }
}

}  // namespace dgrad
