// fp4q_act.h -- the gated operators' activation functions and their derivatives, in fp32.
//
//   silu       g p(g)                                 p the logistic function
//   gelu       g P(g)                                 P the normal distribution's
//   gelu_tanh  g (1 + tanh(c (g + d g^3))) / 2 = g p(2 c (g + d g^3)),   c = sqrt(2 / pi), d = 0.044715
//   relu       max(g, 0), with derivative 0 at 0
//
// With e = exp(-z), p(z) = 1 / (1 + e) and 1 - p(z) = e p(z), so the derivative p (1 - p) has
// no cancellation.  Far from zero e is 0 or infinity and p is 1 or 0, and so are the products with
// g right for every finite g: only an infinite e, and an infinite g where the result has a limit,
// are held to the largest number (0 infinity would be NaN).  (z held to a far value instead would
// leave p at that value's, and g times that of a large g.)  A NaN stays a NaN in every result.
#pragma once

#include <hip/hip_runtime.h>

#include "fp4q_gated.h"

namespace fp4q_act {

constexpr float kMost = 0x1.fffffep127f;

// e^z as 2^t of the rounded t = z log2(e): off by |z| 2^-24 of itself besides the
// instruction's own unit.  Two terms more would take that away, at 0 to 5 % of the gradient kernel's
// time (fp32 gelu 28 %), and no code fewer is off: over 12 seeds of seven cases 0.5 to 1.7 codes in a
// million fall to the other side of a tie than those of 64-bit values, with the terms as without.
// Where |z| is large, e^z or 1 / e^z hardly counts in what is made of it.
__device__ __forceinline__ float exp_of(float z) { return __builtin_amdgcn_exp2f(z * 1.44269504088896340736f); }

struct Logistic {
    float p, q;  // p(z), 1 - p(z)
};
__device__ __forceinline__ Logistic logistic(float z) {
    const float e = exp_of(-z), p = __builtin_amdgcn_rcpf(1.0f + e);
    return {p, __builtin_amdgcn_fmed3f(e, 0.0f, kMost) * p};
}

// Values without infinities, and without the lower one.  (Of a NaN the median is a finite value:
// the factors that these meet are NaN then.)
__device__ __forceinline__ float finite(float v) { return __builtin_amdgcn_fmed3f(v, -kMost, kMost); }
__device__ __forceinline__ float above(float v) { return __builtin_amdgcn_fmed3f(v, -kMost, __builtin_inff()); }

struct Value {
    float act, slope;
};
// The activation and its derivative; what is not used is not computed.
template <int kAct>
__device__ __forceinline__ Value activate(float g) {
    if constexpr (kAct == FP4Q_ACT_SILU) {
        const Logistic s = logistic(g);
        const float act = above(g) * s.p;
        return {act, fmaf(finite(act), s.q, s.p)};
    } else if constexpr (kAct == FP4Q_ACT_GELU) {
        // P(-x) = t Q(t) exp(-x^2 / 2) for x >= 0, t = 1 / (1 + 0.45 x / sqrt 2): Q, of degree 9,
        // fitted to erfcx(x / sqrt 2) / 2 t by least squares of the relative error, reweighted until it
        // is level: 4.8e-8 with the coefficients as they stand here, in fp32, up to x = 30.  One
        // exponential serves P and the density, and P of a far negative g keeps its relative precision.
        const float e = exp_of(-0.5f * g * g);
        g = above(g);
        const float t = __builtin_amdgcn_rcpf(fmaf(0.31819805153394638f, fabsf(g), 1.0f));
        constexpr float kQ[] = {0x1.03fa84p-3f, 0x1.03f9f2p-3f, 0x1.d38016p-4f, 0x1.66ea8ep-4f, 0x1.eb516cp-5f,
                                -0x1.6e5304p-7f, 0x1.23a3bep-4f, -0x1.33cc34p-3f, 0x1.8687b4p-4f, -0x1.5313c0p-6f};
        float q = kQ[9];
#pragma unroll
        for (int i = 8; i >= 0; --i) q = fmaf(q, t, kQ[i]);
        const float low = q * t * e, cdf = g > 0.0f ? 1.0f - low : low;
        return {g * cdf, fmaf(finite(g), 0.39894228040143267794f * e, cdf)};
    } else if constexpr (kAct == FP4Q_ACT_GELU_TANH) {
        constexpr float kTwoC = 1.59576912160573071176f, kD = 0.044715f;
        // |g| > 16 gives |z| > 300, where p is 0 or 1; the square of a larger one could leave fp32's range
        const float near = g > 16.0f ? 16.0f : g < -16.0f ? -16.0f : g, square = near * near;
        const Logistic s = logistic(kTwoC * near * fmaf(kD, square, 1.0f));
        const float slope_z = kTwoC * fmaf(3.0f * kD, square, 1.0f);
        return {above(g) * s.p, fmaf(near * slope_z * s.p, s.q, s.p)};
    } else {
        return {g > 0.0f ? g : g == g ? 0.0f : g, g > 0.0f ? 1.0f : g == g ? 0.0f : g};
    }
}

// Calls f(std::integral_constant<int, activation>) for the activation of that number.
template <typename F>
__host__ __device__ __forceinline__ auto with_act(int act, F &&f) {
    switch (act) {
        case FP4Q_ACT_SILU: return f(std::integral_constant<int, FP4Q_ACT_SILU>{});
        case FP4Q_ACT_GELU: return f(std::integral_constant<int, FP4Q_ACT_GELU>{});
        case FP4Q_ACT_GELU_TANH: return f(std::integral_constant<int, FP4Q_ACT_GELU_TANH>{});
        default: return f(std::integral_constant<int, FP4Q_ACT_RELU>{});
    }
}
inline bool bad_act(int act) { return act < FP4Q_ACT_SILU || act > FP4Q_ACT_RELU; }

}  // namespace fp4q_act
