// owq_act.h -- the activations of the gated feed-forward block and their slopes,
// in fp32.
//   silu       v s(v),  s(v) = 1 / (1 + exp(-v))
//   gelu       v P(v),  P(v) = erfc(-v / sqrt 2) / 2 (the normal distribution; erfc
//              keeps its relative accuracy in the left tail, 1 + erf does not)
//   gelu_tanh  v s(2 c (v + 0.044715 v^3)),  c = sqrt(2 / pi): the tanh form,
//              (1 + tanh t) / 2 = s(2 t)
//   relu       max(v, 0)
// The logistic function uses the hardware's 2^v and reciprocal (one ulp each): its
// relative error is |v| 2^-24 from the rounded exponent plus 2^-22, as large as the
// change of s(v) from the fp32 rounding of v itself; an accurate exp and an IEEE
// division cost four times the instructions, and the two elementwise passes of the
// backward are bound by them. Far out exp overflows to infinity and the quotients to 0: no NaN from finite v
// (|v| < 2^51 for finite fp16 layer inputs, so v^2 stays finite).
#pragma once

#include <type_traits>

#include "owq_device.h"
#include "owq_launch.h"

namespace owq {
namespace {

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTwoC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kCube = 0.044715f;

__device__ __forceinline__ float sigmoid(float v)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * v));
}

template <int ACT>
__device__ __forceinline__ float act_value(float v)
{
    if constexpr (ACT == kActSilu)
        return v * sigmoid(v);
    else if constexpr (ACT == kActGelu)
        return 0.5f * v * erfcf(-v * kSqrtHalf);
    else if constexpr (ACT == kActGeluTanh)
        return v * sigmoid(kTwoC * (v + kCube * v * v * v));
    else
        return fmaxf(v, 0.0f);
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
        const float p = 0.5f * erfcf(-v * kSqrtHalf);
        a = v * p;
        d = p + v * (kInvSqrt2Pi * expf(-0.5f * v * v));
    } else if constexpr (ACT == kActGeluTanh) {
        const float p = sigmoid(kTwoC * (v + kCube * v * v * v));
        a = v * p;
        d = p + v * (p * (1.0f - p)) * (kTwoC * (1.0f + 3.0f * kCube * v * v));
    } else {
        a = fmaxf(v, 0.0f);
        d = v > 0.0f ? 1.0f : 0.0f;
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
