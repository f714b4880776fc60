// The activations of the linear layers and their slopes, in fp32.  `act` is uniform over the grid:
// each function branches on it once for a whole array.
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

// min(|x|, limit), NaN if x is one.
__device__ __forceinline__ float abs_min(float x, float limit)
{
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(fabsf(x)), "f"(limit));
    return y;
}

__device__ __forceinline__ uint64_t f2_both(float x) { return ptx::f2_pack(x, x); }

__device__ __forceinline__ uint64_t f2_ex2(uint64_t x)
{
    float lo, hi;
    ptx::f2_unpack(x, lo, hi);
    return ptx::f2_pack(ptx::ex2(lo), ptx::ex2(hi));
}

__device__ __forceinline__ uint64_t f2_rcp(uint64_t x)
{
    float lo, hi;
    ptx::f2_unpack(x, lo, hi);
    return ptx::f2_pack(rcp_approx(lo), rcp_approx(hi));
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluK = 0.79788456080286536f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// erfc(x) / 2 for x >= 0 in the form of the rational approximations 7.1.25 to 7.1.28 of Abramowitz and
// Stegun's Handbook of Mathematical Functions,
//   erfc(x) / 2 = (c1 t + c2 t^2 + ... + c6 t^6) exp(-x^2), t = 1 / (1 + p x).
// GELU left of zero is this small quantity itself, so it has to be right relative to its value as well, which
// the handbook's coefficients are not (0.4 % at z = -6, 1.5 % at -9).  These are fitted (reweighted least
// squares in 64 bits until the largest error stands still) for an absolute error of at most 6e-8 and a relative
// one of at most 2e-4 at once, up to x = 9.4; in fp32, GELU for -13 <= z < 0 is off by at most 1.9e-4 of its
// value, an eighth of half a bf16 step at most, and by at most 7.2e-8 (1 + |z|) anywhere.
constexpr float kErfP = 0.58f, kErfC1 = 0.1623907006652872f, kErfC2 = 0.1801755865978446f,
                kErfC3 = 0.05218518602756604f, kErfC4 = 0.28861909495540805f, kErfC5 = -0.23919958357453605f,
                kErfC6 = 0.05582905727140084f;
constexpr float kSqrtHalf = 0.70710678118654752f;

// z <- act(z) for pairs of values (packed fp32 arithmetic: two multiply-adds an instruction, which
// keeps the epilogues that use it ahead of the tensor cores).
template <int NP>
__device__ __forceinline__ void activate(uint64_t (&z)[NP], int act)
{
    using namespace ptx;
    if (act == ATTN_ACT_GELU) {
        // z Phi(z) = max(z, 0) - |z| erfc(|z| / sqrt 2) / 2; |z| stops at 100, where the second term
        // has long vanished, so that an infinity keeps its value
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            float lo, hi;
            f2_unpack(z[i], lo, hi);
            const uint64_t a = f2_pack(abs_min(lo, 100.f), abs_min(hi, 100.f));
            const uint64_t t = f2_rcp(fma_f32x2(a, f2_both(kErfP * kSqrtHalf), f2_both(1.f)));
            const uint64_t e = f2_ex2(mul_f32x2(mul_f32x2(a, f2_both(-0.5f * kLog2e)), a));
            uint64_t s = fma_f32x2(t, f2_both(-kErfC6), f2_both(-kErfC5));
            s = fma_f32x2(t, s, f2_both(-kErfC4));
            s = fma_f32x2(t, s, f2_both(-kErfC3));
            s = fma_f32x2(t, s, f2_both(-kErfC2));
            s = fma_f32x2(t, s, f2_both(-kErfC1));
            s = mul_f32x2(mul_f32x2(t, s), e);
            z[i] = fma_f32x2(a, s, f2_pack(fmaxf(lo, 0.f), fmaxf(hi, 0.f)));
        }
    } else if (act == ATTN_ACT_GELU_TANH) {
        // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const uint64_t w = fma_f32x2(mul_f32x2(z[i], z[i]), f2_both(-2.f * kLog2e * kGeluK * kGeluA),
                                         f2_both(-2.f * kLog2e * kGeluK));
            z[i] = mul_f32x2(z[i], f2_rcp(add_f32x2(f2_ex2(mul_f32x2(z[i], w)), f2_both(1.f))));
        }
    } else if (act == ATTN_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < NP; ++i)
            z[i] = mul_f32x2(z[i], f2_rcp(add_f32x2(f2_ex2(mul_f32x2(z[i], f2_both(-kLog2e))), f2_both(1.f))));
    } else if (act == ATTN_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            float lo, hi;
            f2_unpack(z[i], lo, hi);
            asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(lo));
            asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(hi));
            z[i] = f2_pack(lo, hi);
        }
    }
}

__device__ __forceinline__ float sigmoid(float x) { return rcp_approx(1.f + ptx::ex2(-kLog2e * x)); }

// d <- d act'(z).
template <int N>
__device__ __forceinline__ void times_slope(float (&d)[N], const float (&z)[N], int act)
{
    if (act == ATTN_ACT_GELU) {
        // Phi(z) + z phi(z), with Phi(-a) = 1 - Phi(a)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float a = abs_min(z[i], 100.f);
            const float t = rcp_approx(fmaf(a, kErfP * kSqrtHalf, 1.f)), e = ptx::ex2(-0.5f * kLog2e * a * a);
            float s = fmaf(t, kErfC6, kErfC5);
            s = fmaf(t, s, kErfC4);
            s = fmaf(t, s, kErfC3);
            s = fmaf(t, s, kErfC2);
            s = fmaf(t, s, kErfC1);
            // slope(a) = 1 - tail for z >= 0, tail for z < 0
            const float tail = e * fmaf(t, s, -0.39894228040143268f * a);
            d[i] *= z[i] >= 0.f ? 1.f - tail : tail;
        }
    } else if (act == ATTN_ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float x = z[i], q = x * x, p = sigmoid(2.f * kGeluK * x * fmaf(kGeluA, q, 1.f)), r = p * (1.f - p);
            // r is 0 where the square may overflow
            d[i] *= r == 0.f ? p : fmaf(x * r, 2.f * kGeluK * fmaf(3.f * kGeluA, q, 1.f), p);
        }
    } else if (act == ATTN_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float p = sigmoid(z[i]);
            d[i] *= p * fmaf(z[i], 1.f - p, 1.f);
        }
    } else if (act == ATTN_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = z[i] > 0.f ? d[i] : 0.f;
    }
}

}  // namespace attn
