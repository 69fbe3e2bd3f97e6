// gate_act.cuh -- the gate's activations and their derivatives, in fp32, two elements at a
// time (packed FP32 instructions; the exponential and reciprocal units take one).
//
// With s(v) = 1/(1 + exp(-v)) and P the normal distribution:
//   silu       g s(g)                       s (1 + g (1 - s))
//   gelu       g P(g)                       P + g exp(-g^2/2)/sqrt(2 pi)
//   gelu_tanh  g s(2v), v = sqrt(2/pi)(g + 0.044715 g^3)   (the same as g(1 + tanh v)/2)
//                                           s + 2 g s (1 - s) dv/dg
//   relu       max(g, 0)                    g > 0
//   sigmoid    s(g)                         s(g) s(-g)
//   none       g                            1                 (group norm only)
// The forms keep their relative precision for large negative g, where 1 + tanh and
// 1 + erf cancel, and sigmoid's derivative for large positive g, where 1 - s does (at
// g = 12 s (1 - s) is off by 1%, from 17 on it is 0).  P's tail is
// t 2^(p(t) - g^2/(2 ln 2)), t = 1/(1 + 0.29|g|), with p a polynomial of degree 8 fitted to
// log2(erfcx(|g|/sqrt 2)/(2t)) by weighted least squares on Chebyshev nodes (relative error
// 2.5e-7; 8e-7 with fp32 rounding for |g| < 4).
// ex2 and rcp are the hardware's approximations (about 2^-22), far below a 16-bit
// result's half step.  With the general-purpose exp, division and erfc the epilogue took
// longer than the tile's MMAs: 32768 rows, 768 to 2048 channels, bf16 silu 149 us, gelu
// 203; with these forms 144 and 155.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace dgrad {

enum GateAct : int { kSilu = 0, kGelu = 1, kGeluTanh = 2, kRelu = 3, kSigmoid = 4, kNoAct = 5 };

__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }

__device__ __forceinline__ float2 ex2_pair(float2 v)
{
    float2 r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(v.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(v.y));
    return r;
}

__device__ __forceinline__ float2 rcp_pair(float2 v)
{
    float2 r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(v.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(v.y));
    return r;
}

// 1/(1 + 2^w): s(v) for w = -v log2(e).
__device__ __forceinline__ float2 logistic2(float2 w) { return rcp_pair(__fadd2_rn(ex2_pair(w), splat(1.0f))); }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTanhA = 0.7978845608028654f;             // sqrt(2/pi)
constexpr float kTanhB = 0.7978845608028654f * 0.044715f;

// P(g), and e = 2^(-g^2/(2 ln 2)) = exp(-g^2/2) when E.
template <bool E>
__device__ __forceinline__ float2 normal_cdf(float2 g, float2* e)
{
    const float2 a = make_float2(fabsf(g.x), fabsf(g.y));
    const float2 t = rcp_pair(ffma2(a, splat(0.29f), splat(1.0f)));
    float2 p = splat(-0.27778888f);
    p = ffma2(p, t, splat(1.1824034f));
    p = ffma2(p, t, splat(-1.7660975f));
    p = ffma2(p, t, splat(1.0227866f));
    p = ffma2(p, t, splat(-0.42359963f));
    p = ffma2(p, t, splat(0.34500575f));
    p = ffma2(p, t, splat(0.58516502f));
    p = ffma2(p, t, splat(1.4437800f));
    p = ffma2(p, t, splat(-3.1116550f));
    const float2 h = __fmul2_rn(g, splat(-0.5f * kLog2e));
    const float2 q = __fmul2_rn(t, ex2_pair(ffma2(h, g, p)));
    if constexpr (E) *e = ex2_pair(__fmul2_rn(h, g));
    return make_float2(g.x > 0.f ? 1.0f - q.x : q.x, g.y > 0.f ? 1.0f - q.y : q.y);
}

template <int ACT>
__device__ __forceinline__ float2 gate_act(float2 g)
{
    if constexpr (ACT == kSilu) {
        return __fmul2_rn(g, logistic2(__fmul2_rn(g, splat(-kLog2e))));
    } else if constexpr (ACT == kGelu) {
        return __fmul2_rn(g, normal_cdf<false>(g, nullptr));
    } else if constexpr (ACT == kGeluTanh) {
        const float2 c = ffma2(__fmul2_rn(g, splat(-2.0f * kLog2e * kTanhB)), g, splat(-2.0f * kLog2e * kTanhA));
        return __fmul2_rn(g, logistic2(__fmul2_rn(g, c)));
    } else if constexpr (ACT == kRelu) {
        return make_float2(g.x <= 0.f ? 0.f : g.x, g.y <= 0.f ? 0.f : g.y);   // NaN stays
    } else if constexpr (ACT == kNoAct) {
        return g;
    } else {
        return logistic2(__fmul2_rn(g, splat(-kLog2e)));
    }
}

// a = act(g), d = act'(g).
template <int ACT>
__device__ __forceinline__ void gate_act_grad(float2 g, float2& a, float2& d)
{
    if constexpr (ACT == kSilu) {
        const float2 s = logistic2(__fmul2_rn(g, splat(-kLog2e)));
        a = __fmul2_rn(g, s);
        const float2 rest = ffma2(s, splat(-1.0f), splat(1.0f));
        d = __fmul2_rn(s, ffma2(g, rest, splat(1.0f)));
    } else if constexpr (ACT == kGelu) {
        float2 e;
        const float2 p = normal_cdf<true>(g, &e);
        a = __fmul2_rn(g, p);
        d = ffma2(__fmul2_rn(g, splat(0.3989422804014327f)), e, p);
    } else if constexpr (ACT == kGeluTanh) {
        const float2 g2 = __fmul2_rn(g, g);
        const float2 s = logistic2(__fmul2_rn(g, ffma2(g2, splat(-2.0f * kLog2e * kTanhB), splat(-2.0f * kLog2e * kTanhA))));
        float2 dv2 = ffma2(g2, splat(6.0f * kTanhB), splat(2.0f * kTanhA));
        dv2 = make_float2(fminf(dv2.x, 1e30f), fminf(dv2.y, 1e30f));   // finite: s (1 - s) is 0 there
        a = __fmul2_rn(g, s);
        const float2 rest = ffma2(s, splat(-1.0f), splat(1.0f));
        d = ffma2(__fmul2_rn(a, rest), dv2, s);   // 2 a would pass fp32's largest value before rest is 0
    } else if constexpr (ACT == kRelu) {
        a = gate_act<kRelu>(g);
        d = make_float2(g.x > 0.f ? 1.0f : 0.f, g.y > 0.f ? 1.0f : 0.f);
    } else if constexpr (ACT == kNoAct) {
        a = g;
        d = splat(1.0f);
    } else {
        const float2 x = ex2_pair(__fmul2_rn(make_float2(fabsf(g.x), fabsf(g.y)), splat(-kLog2e)));
        const float2 r = rcp_pair(__fadd2_rn(x, splat(1.0f))), o = __fmul2_rn(x, r);   // s(|g|), s(-|g|)
        a = make_float2(g.x > 0.f ? r.x : o.x, g.y > 0.f ? r.y : o.y);
        d = __fmul2_rn(r, o);
    }
}

// Calls f with the activation as a compile-time constant: the branch lies outside the
// element loops, so that the elements' long-latency instructions overlap.
template <typename F>
__device__ __forceinline__ void with_act(int act, F f)
{
    switch (act) {
    case kSilu: f(std::integral_constant<int, kSilu>{}); break;
    case kGelu: f(std::integral_constant<int, kGelu>{}); break;
    case kGeluTanh: f(std::integral_constant<int, kGeluTanh>{}); break;
    case kRelu: f(std::integral_constant<int, kRelu>{}); break;
    default: f(std::integral_constant<int, kSigmoid>{}); break;
    }
}

}  // namespace dgrad
