// Activations of the gated feed-forward operators and their derivatives, in
// float32, and the 16-bit conversions around them.
#pragma once
#include "../device.hpp"
#include "ffn.hpp"

namespace bsg {
namespace ffn {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// sigmoid(t) and 1 - sigmoid(t) from one exponential of -|t|, which never
// overflows: with e = exp(-|t|) and r = 1 / (1 + e), the two are r and e*r.
// (1 - s formed by subtraction would lose its digits where s is near 1.)
struct Sig {
    float s, c;
};
__device__ __forceinline__ Sig sigmoid2(float t)
{
    const float e = __builtin_amdgcn_exp2f(-1.44269504f * fabsf(t));
    const float r = __builtin_amdgcn_rcpf(1.0f + e), er = e * r;
    return t >= 0.0f ? Sig{r, er} : Sig{er, r};
}

// tanh-form GELU: 0.5 x (1 + tanh z) = x sigmoid(2z) with
// z = sqrt(2/pi) (x + 0.044715 x^3).  x^2 is held at 1e37, past which the
// sigmoid is 0 or 1 anyway, so that nothing below multiplies 0 by infinity.
constexpr float kGelu2C = 1.59576912f, kGeluA = 0.044715f;   // 2 sqrt(2/pi)

// act(x)
template <int ACT>
__device__ __forceinline__ float act_value(float x)
{
    if constexpr (ACT == ACT_SILU) return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * x));
    else if constexpr (ACT == ACT_RELU) return x < 0.0f ? 0.0f : x;     // NaN stays NaN
    else {
        const float x2 = fminf(x * x, 1e37f);
        const float t = kGelu2C * x * (1.0f + kGeluA * x2);
        return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * t));
    }
}

// act(x) and act'(x)
struct ActGrad {
    float v, d;
};
template <int ACT>
__device__ __forceinline__ ActGrad act_grad(float x)
{
    if constexpr (ACT == ACT_SILU) {
        const Sig p = sigmoid2(x);
        const float v = x * p.s;
        return {v, p.s + v * p.c};
    } else if constexpr (ACT == ACT_RELU) {
        return {x < 0.0f ? 0.0f : x, x > 0.0f ? 1.0f : 0.0f};
    } else {
        const float x2 = fminf(x * x, 1e37f);
        const Sig p = sigmoid2(kGelu2C * x * (1.0f + kGeluA * x2));
        const float v = x * p.s;
        return {v, p.s + v * p.c * kGelu2C * (1.0f + 3.0f * kGeluA * x2)};
    }
}

// f(std::integral_constant<int, ACT>) for a run-time activation
template <class F>
auto with_act(int act, F &&f)
{
    switch (act) {
    case ACT_SILU: return f(std::integral_constant<int, ACT_SILU>{});
    case ACT_RELU: return f(std::integral_constant<int, ACT_RELU>{});
    default: return f(std::integral_constant<int, ACT_GELU_TANH>{});
    }
}

// 16-bit pairs (DT_F16 / DT_BF16), low half first
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    if constexpr (DT == DT_BF16) return pack2_bf16(a, b);
    else return pack2_f16(a, b);
}
template <int DT>
__device__ __forceinline__ float lo16(uint32_t w)
{
    if constexpr (DT == DT_BF16) return __uint_as_float(w << 16);
    else return (float)__builtin_bit_cast(f16x2_t, w).x;
}
template <int DT>
__device__ __forceinline__ float hi16(uint32_t w)
{
    if constexpr (DT == DT_BF16) return __uint_as_float(w & 0xFFFF0000u);
    else return (float)__builtin_bit_cast(f16x2_t, w).y;
}

}  // namespace ffn
}  // namespace bsg
