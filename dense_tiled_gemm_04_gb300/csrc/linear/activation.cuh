// The activations of the linear-layer kernels and their derivatives, in fp32.
//
//   act        value                          slope
//   kRelu      z < 0 ? 0 : z                  z <= 0 ? 0 : 1
//   kGelu      z Phi(z)                       Phi(z) + z phi(z)
//   kGeluTanh  z s(2u)                        s + z s (1 - s) 2u',  2u = z (c0 + c1 z^2)
//   kSilu      z s(z)                         s (1 + z (1 - s))
// with Phi, phi the normal distribution and density and s the logistic function.
//
// The epilogues are bound by instruction issue (a 128 x 256 tile over a contraction of 1024 leaves 32 issue slots per
// element), so every form here takes 15 instructions or fewer, two of them on the special-function unit:
//  * s(t) = 1 / (1 + 2^(-t log2 e)) from the approximate exponential and reciprocal (about an ulp each, three
//    decimal digits under the rounding to 16 bits).  z s(t) keeps its relative precision for negative z, where
//    1 + tanh(u) would cancel.
//  * Phi(-a) = e^(-a^2/2) h(a) for a >= 0, with h(a) = erfcx(a / sqrt 2) / 2 = t Q(t), t = 1 / (1 + 0.3 a): Q is a
//    polynomial of degree 7, fitted to the least largest relative error over a in [0, 14] by iteratively reweighted
//    least squares (Lawson's method): 1.5e-7, 5e-7 as evaluated in fp32.  Both the value, max(z, 0) - a Phi(-a),
//    and the slope, u or 1 - u with u = e^(-a^2/2) (h - a / sqrt(2 pi)), share it.  erff and the exponential took 60
//    instructions more per slope: dgrad 16384 x 1024 x 8192 spent 678 us with gelu and 373 us with relu.
// Arguments are clamped to ranges outside which values and slopes equal their limits in fp32, so infinities give
// the limits; the clamps let NaN pass.
#pragma once

#include <cstdint>

namespace dtg {
namespace linear {

constexpr int kActNone = 0, kRelu = 1, kGelu = 2, kGeluTanh = 3, kSilu = 4;  // gemm_act_t

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhC0 = 1.5957691216057308f;    // 2 sqrt(2/pi)
constexpr float kTanhC1 = 0.071354816272600249f;  // 2 sqrt(2/pi) 0.044715

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// max and min that return NaN when an argument is NaN.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

__device__ __forceinline__ float min_nan(float a, float b)
{
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// e^(-a^2/2) with z^2 = a^2 (0 for infinities), and h(a) above for a in [0, 14].
__device__ __forceinline__ float gauss(float z) { return ex2(z * z * (-0.5f * kLog2e)); }

__device__ __forceinline__ float half_erfcx(float a)
{
    const float t = rcp(fmaf(0.3f, a, 1.0f));
    float q = 0.03567477688193321f;
    q = fmaf(q, t, -0.15720310807228088f);
    q = fmaf(q, t, 0.20635353028774261f);
    q = fmaf(q, t, -0.05368367210030556f);
    q = fmaf(q, t, 0.12856164574623108f);
    q = fmaf(q, t, 0.09991348534822464f);
    q = fmaf(q, t, 0.12075395882129669f);
    q = fmaf(q, t, 0.11962930113077164f);
    return q * t;
}

template <int ACT>
__device__ __forceinline__ float act_value(float z)
{
    if constexpr (ACT == kRelu) return max_nan(z, 0.0f);
    if constexpr (ACT == kGelu) {
        const float a = fminf(fabsf(z), 14.0f);  // a NaN z reaches the result through gauss(z)
        return fmaf(-a * gauss(z), half_erfcx(a), fmaxf(z, 0.0f));
    }
    if constexpr (ACT == kGeluTanh) {
        const float c = max_nan(z, -12.0f);
        return c * rcp(1.0f + ex2(c * fmaf(-kTanhC1 * kLog2e * c, c, -kTanhC0 * kLog2e)));
    }
    if constexpr (ACT == kSilu) {
        const float c = max_nan(z, -100.0f);
        return c * rcp(1.0f + ex2(-kLog2e * c));
    }
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z)
{
    if constexpr (ACT == kRelu) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);  // NaN stays NaN
    if constexpr (ACT == kGelu) {
        const float a = fminf(fabsf(z), 14.0f);
        const float u = gauss(z) * fmaf(-kInvSqrt2Pi, a, half_erfcx(a));
        return z < 0.0f ? u : 1.0f - u;
    }
    if constexpr (ACT == kGeluTanh) {
        const float c = max_nan(min_nan(z, 12.0f), -12.0f);
        const float q = c * c;
        const float s = rcp(1.0f + ex2(c * fmaf(-kTanhC1 * kLog2e, q, -kTanhC0 * kLog2e)));
        return fmaf(c * s * (1.0f - s), fmaf(3.0f * kTanhC1, q, kTanhC0), s);
    }
    if constexpr (ACT == kSilu) {
        const float c = max_nan(min_nan(z, 100.0f), -100.0f);
        const float s = rcp(1.0f + ex2(-kLog2e * c));
        return s * fmaf(c, 1.0f - s, 1.0f);
    }
    return 1.0f;
}

// Runs f<ACT>() for the activation of a launch (uniform over the grid).
#define DTG_ACT_SWITCH(act, STATEMENT)                              \
    switch (act) {                                                  \
    case kRelu: { constexpr int ACT = kRelu; STATEMENT; } break;          \
    case kGelu: { constexpr int ACT = kGelu; STATEMENT; } break;          \
    case kGeluTanh: { constexpr int ACT = kGeluTanh; STATEMENT; } break;  \
    case kSilu: { constexpr int ACT = kSilu; STATEMENT; } break;          \
    default: { constexpr int ACT = kActNone; STATEMENT; } break;          \
    }

}  // namespace linear
}  // namespace dtg
