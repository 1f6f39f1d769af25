// activation.h -- the gated block's activations and their derivatives in FP32.
//
// act(g) is SiLU, g / (1 + exp(-g)); the tanh GeLU in its sigmoid form,
// g / (1 + exp(-2 sqrt(2/pi) (g + 0.044715 g^3))); or the erf GeLU,
// g Phi(g) with Phi(g) = erfc(-g / sqrt 2) / 2 (the complementary function keeps
// Phi's relative precision where it is small).  The block works on its FP32 sums
// and rounds once, unlike the epilogue program, whose steps each round to the
// element type.  exp and the reciprocal are the hardware's (about 1 ulp of FP32,
// 2^13 times finer than the words' last place); their special values give the
// formulas' own: a sum of -inf gives NaN (-inf * 0), as -inf / inf does.
#pragma once

#include "common.h"

namespace lin {

// 1 / (1 + exp(-z))
__device__ inline float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

constexpr float kGeluA = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;
constexpr float kRsqrt2 = 0.70710678118654752f;
constexpr float kRsqrt2Pi = 0.39894228040143268f;

__device__ inline float gated_act(int act, float g) {
    if (act == kEpiGeluErf) return g * (0.5f * erfcf(-g * kRsqrt2));
    const float z = act == kEpiGeluTanh ? kGeluA * (g + kGeluB * (g * g * g)) : g;
    return g * sigmoid(z);
}

// act(g) and act'(g).
__device__ inline void gated_act_grad(int act, float g, float& a, float& d) {
    if (act == kEpiGeluErf) {
        const float p = 0.5f * erfcf(-g * kRsqrt2);
        a = g * p;
        d = p + g * (kRsqrt2Pi * __expf(-0.5f * g * g));
        return;
    }
    float z = g, dz = 1.f;
    if (act == kEpiGeluTanh) {
        z = kGeluA * (g + kGeluB * (g * g * g));
        dz = kGeluA * (1.f + 3.f * kGeluB * fminf(g * g, 1e30f));   // finite: far out it meets a sigmoid of 0
    }
    const float s = sigmoid(z);
    a = g * s;
    // s' = s (1 - s), with 1 - s taken as the other sigmoid: no cancellation
    d = s + a * (sigmoid(-z) * dz);
}

}  // namespace lin
