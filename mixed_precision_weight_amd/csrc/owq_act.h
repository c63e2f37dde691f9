// owq_act.h -- the activations of the gated feed-forward block and their slopes,
// in fp32.
//   silu       v s(v),  s(v) = 1 / (1 + exp(-v))
//   gelu       v P(v),  P(v) the normal distribution, with its relative accuracy in
//              the left tail too (see normal)
//   gelu_tanh  v s(2 c (v + 0.044715 v^3)),  c = sqrt(2 / pi): the tanh form,
//              (1 + tanh t) / 2 = s(2 t)
//   relu       max(v, 0)
// All four keep a NaN (relu compares: the hardware's maximum of NaN and 0 is 0), in the
// value and in the slope, so that a step that diverged shows in its gradients.
// The logistic function uses the hardware's 2^v and reciprocal (one ulp each): its
// relative error is |v| 2^-24 from the rounded exponent plus 2^-22, as large as the
// change of s(v) from the fp32 rounding of v itself; an accurate exp and an IEEE
// division cost four times the instructions, and the two elementwise passes of the
// backward are bound by them. Far out exp overflows to infinity and the quotients to
// 0: no NaN from finite v. (|v| < 2^51 for finite fp16 layer inputs, so v^2 stays
// finite; the cubic of gelu_tanh is infinite from about |v| = 2^44, where s is 0 or 1.)
#pragma once

#include <type_traits>

#include "owq_device.h"
#include "owq_launch.h"

namespace owq {
namespace {

constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTwoC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kCube = 0.044715f;

__device__ __forceinline__ float sigmoid(float v)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * v));
}

// p = P(v), the normal distribution, and e = exp(-v^2 / 2). With x = |v|,
// P(-x) = e q(x), and q = P(-x) exp(x^2 / 2) is smooth: a polynomial of degree 10 in
// t = 1 / (1 + x / 4), without constant term (q falls as 1 / x). Its coefficients are a
// reweighted least-squares fit over x in [0, 200]; as fp32 constants its largest
// relative error is 2^-23.5 (at x = 0.054). x^2 and its product with log2(e) / 2 are
// carried with their rounding errors, which correct the hardware's 2^v, so that the tail
// keeps p's relative error at 2^-20.5 (most of it the Horner sum's) up to x = 13.1; p is
// subnormal from x = 12.95 on. From x = 13.22 on the hardware's 2^v gives 0 for its
// subnormal results, and so is the tail, where P(-x) < 2^-131. With erfc and exp of the compiler's library, and their branches, the elementwise passes of a
// training step of 2048 tokens, 2 x 11008 x 4096, took 103 + 104 us, now 85 + 81.
__device__ __forceinline__ void normal(float v, float& p, float& e)
{
    constexpr float kHi = 0.72134752f, kLo = (float)(0.72134752044448170368 - (double)kHi);  // log2(e) / 2
    constexpr float kLn2 = 0.69314718f;
    const float x = fminf(fabsf(v), 16.0f);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(x, 0.25f, 1.0f));
    float q = 0.0203713309f;
    q = __builtin_fmaf(q, t, -0.0834895819f);
    q = __builtin_fmaf(q, t, 0.100448258f);
    q = __builtin_fmaf(q, t, -0.0366198272f);
    q = __builtin_fmaf(q, t, 0.0666298792f);
    q = __builtin_fmaf(q, t, 0.0579195209f);
    q = __builtin_fmaf(q, t, 0.0818264955f);
    q = __builtin_fmaf(q, t, 0.0934405178f);
    q = __builtin_fmaf(q, t, 0.0997378305f);
    q = __builtin_fmaf(q, t, 0.0997355431f);
    const float s = x * x, ds = __builtin_fmaf(x, x, -s);
    const float y = s * kHi;
    const float dy = __builtin_fmaf(ds, kHi, __builtin_fmaf(s, kLo, __builtin_fmaf(s, kHi, -y)));
    const float e0 = __builtin_amdgcn_exp2f(-y);
    e = __builtin_fmaf(e0 * -kLn2, dy, e0);
    const float tail = q * t * e;
    p = v < 0.0f ? tail : 1.0f - tail;
}

template <int ACT>
__device__ __forceinline__ float act_value(float v)
{
    if constexpr (ACT == kActSilu)
        return v * sigmoid(v);
    else if constexpr (ACT == kActGelu) {
        float p, e;
        normal(v, p, e);
        return v * p;
    } else if constexpr (ACT == kActGeluTanh)
        return v * sigmoid(kTwoC * (v + kCube * v * v * v));
    else
        return v <= 0.0f ? 0.0f : v;
}

// value and slope at v
template <int ACT>
__device__ __forceinline__ void act_both(float v, float& a, float& d)
{
    if constexpr (ACT == kActSilu) {
        const float p = sigmoid(v);
        a = v * p;
        d = p * (1.0f + v * (1.0f - p));
    } else if constexpr (ACT == kActGelu) {
        float p, e;
        normal(v, p, e);
        a = v * p;
        d = p + v * (kInvSqrt2Pi * e);
    } else if constexpr (ACT == kActGeluTanh) {
        const float p = sigmoid(kTwoC * (v + kCube * v * v * v));
        a = v * p;
        d = p + v * (p * (1.0f - p)) * (kTwoC * (1.0f + 3.0f * kCube * v * v));
    } else {
        a = v <= 0.0f ? 0.0f : v;
        d = v > 0.0f ? 1.0f : a;
    }
}

// f(integral constant of act): the activation as a compile-time value, chosen in
// the kernel (uniform) or by the host
template <typename F>
__device__ __forceinline__ void with_act(int act, F f)
{
    switch (act) {
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
    default: f(std::integral_constant<int, kActRelu>{}); break;
    }
}

template <typename F>
void for_act(int act, F f)
{
    switch (act) {
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
    default: f(std::integral_constant<int, kActRelu>{}); break;
    }
}

}  // namespace
}  // namespace owq
