// The activations of the linear layers and their slopes, in fp32.
#pragma once

#include "attn.h"
#include "ptx.cuh"

namespace attn {

__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + exp(-x)): two MUFU operations, relative error a few 2^-23.
__device__ __forceinline__ float sigmoid(float x) { return rcp_approx(1.f + ptx::ex2(-kLog2e * x)); }

// The normal distribution function, Phi(z) = erfc(-z / sqrt 2) / 2, by the rational approximation
// 7.1.26 of Abramowitz and Stegun's Handbook of Mathematical Functions:
//   erfc(x) = (a1 t + a2 t^2 + ... + a5 t^5) exp(-x^2) + e, t = 1 / (1 + p x), x >= 0, |e| <= 1.5e-7,
// far below the bf16 rounding of what it multiplies.  `density` gets exp(-z^2 / 2).
__device__ __forceinline__ float normal_cdf(float z, float &density)
{
    const float x = fabsf(z) * 0.70710678118654752f;
    const float t = rcp_approx(fmaf(0.3275911f, x, 1.f));
    density = ptx::ex2(-kLog2e * x * x);
    float s = fmaf(t, 1.061405429f, -1.453152027f);
    s = fmaf(t, s, 1.421413741f);
    s = fmaf(t, s, -0.284496736f);
    s = fmaf(t, s, 0.254829592f);
    const float half_erfc = 0.5f * t * s * density;
    return z >= 0.f ? 1.f - half_erfc : half_erfc;
}

constexpr float kGeluK = 0.79788456080286536f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// act(z).  `act` is uniform over the grid, so the branch costs one predicate.
__device__ __forceinline__ float activate(float z, int act)
{
    float e;
    switch (act) {
    case ATTN_ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);
    case ATTN_ACT_GELU: return z * normal_cdf(z, e);
    // (1 + tanh u) / 2 = sigmoid(2 u)
    case ATTN_ACT_GELU_TANH: return z * sigmoid(2.f * kGeluK * z * fmaf(kGeluA * z, z, 1.f));
    case ATTN_ACT_SILU: return z * sigmoid(z);
    default: return z;
    }
}

// act'(z).
__device__ __forceinline__ float act_slope(float z, int act)
{
    switch (act) {
    case ATTN_ACT_RELU: return z > 0.f ? 1.f : 0.f;
    case ATTN_ACT_GELU: {
        float e;
        const float cdf = normal_cdf(z, e);
        return fmaf(z * 0.39894228040143268f, e, cdf);   // Phi(z) + z phi(z)
    }
    case ATTN_ACT_GELU_TANH: {
        const float p = sigmoid(2.f * kGeluK * z * fmaf(kGeluA * z, z, 1.f)), r = p * (1.f - p);
        // r is 0 where z^2 may overflow
        return r == 0.f ? p : fmaf(z * r, 2.f * kGeluK * fmaf(3.f * kGeluA * z, z, 1.f), p);
    }
    case ATTN_ACT_SILU: {
        const float p = sigmoid(z);
        return p * fmaf(z, 1.f - p, 1.f);
    }
    default: return 1.f;
    }
}

}  // namespace attn
