// The activations of the linear-layer kernels and their derivatives, in fp32.
//
//   act        value                          slope
//   kRelu      z < 0 ? 0 : z                  z <= 0 ? 0 : 1
//   kGelu      z Phi(z)                       Phi(z) + z phi(z)
//   kGeluTanh  z s(2u)                        s + z s (1 - s) 2u',  2u = z (c0 + c1 z^2)
//   kSilu      z s(z)                         s (1 + z (1 - s))
// with Phi, phi the normal distribution and density and s the logistic function.
//
// A 128 x 256 tile over a contraction of 1024 leaves 32 issue slots per element for the whole epilogue, so
// every form here works on pairs of values and takes 12 slots per value or fewer, two of them on the special-function unit:
//  * s(t) = 1 / (1 + 2^(-t log2 e)) from the approximate exponential and reciprocal (about an ulp each, three
//    decimal digits under the rounding to 16 bits).  z s(t) keeps its relative precision for negative z, where
//    1 + tanh(u) would cancel.
//  * Phi(-a) = e^(-a^2/2) h(a) for a >= 0, with h(a) = erfcx(a / sqrt 2) / 2 = t Q(t), t = 1 / (1 + 0.3 a): Q is a
//    polynomial of degree 7, fitted to the least largest relative error over a in [0, 14] by iteratively reweighted
//    least squares (Lawson's method): 1.5e-7, 5e-7 as evaluated in fp32.  Both the value, max(z, 0) - a Phi(-a),
//    and the slope, u or 1 - u with u = e^(-a^2/2) (h - a / sqrt(2 pi)), share it.  With erff and the
//    exponential dgrad 16384 x 1024 x 8192 took 678 us, with the shared polynomial 398 us.
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

// Two fp32 values in a 64-bit register, and the instructions that do two operations at once: they
// halve the issue slots of the multiplies and adds, which leaves the others to the unpaired instructions.
typedef uint64_t f32x2;

__device__ __forceinline__ f32x2 pair(float lo, float hi)
{
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ f32x2 both(float x) { return pair(x, x); }

__device__ __forceinline__ void split(f32x2 v, float& lo, float& hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// f of each half.
template <class F>
__device__ __forceinline__ f32x2 each(f32x2 v, F f)
{
    float lo, hi;
    split(v, lo, hi);
    return pair(f(lo), f(hi));
}

// 1 / (1 + 2^m)
__device__ __forceinline__ f32x2 logistic2(f32x2 m)
{
    return each(add2(each(m, [](float x) { return ex2(x); }), both(1.0f)), [](float x) { return rcp(x); });
}

// e^(-z^2/2) (0 for infinities).
__device__ __forceinline__ f32x2 gauss2(f32x2 z)
{
    return each(mul2(mul2(z, both(-0.5f * kLog2e)), z), [](float x) { return ex2(x); });
}

// h(a) above for -a in [-14, 0].
__device__ __forceinline__ f32x2 half_erfcx2(f32x2 minus_a)
{
    const f32x2 t = each(fma2(minus_a, both(-0.3f), both(1.0f)), [](float x) { return rcp(x); });
    f32x2 q = both(0.03567477688193321f);
    q = fma2(q, t, both(-0.15720310807228088f));
    q = fma2(q, t, both(0.20635353028774261f));
    q = fma2(q, t, both(-0.05368367210030556f));
    q = fma2(q, t, both(0.12856164574623108f));
    q = fma2(q, t, both(0.09991348534822464f));
    q = fma2(q, t, both(0.12075395882129669f));
    q = fma2(q, t, both(0.11962930113077164f));
    return mul2(q, t);
}

// -min(|z|, 14); a NaN becomes -14 (it reaches the results through gauss2).
__device__ __forceinline__ f32x2 minus_abs14(f32x2 z)
{
    return each(z, [](float x) { return fmaxf(-fabsf(x), -14.0f); });
}

template <int ACT>
__device__ __forceinline__ f32x2 act_value2(f32x2 z)
{
    if constexpr (ACT == kRelu) return each(z, [](float x) { return max_nan(x, 0.0f); });
    if constexpr (ACT == kGelu) {
        const f32x2 na = minus_abs14(z);
        return fma2(mul2(na, gauss2(z)), half_erfcx2(na), each(z, [](float x) { return fmaxf(x, 0.0f); }));
    }
    if constexpr (ACT == kGeluTanh) {
        const f32x2 c = each(z, [](float x) { return max_nan(x, -12.0f); });
        return mul2(c, logistic2(mul2(c, fma2(mul2(c, c), both(-kTanhC1 * kLog2e), both(-kTanhC0 * kLog2e)))));
    }
    if constexpr (ACT == kSilu) {
        const f32x2 c = each(z, [](float x) { return max_nan(x, -100.0f); });
        return mul2(c, logistic2(mul2(c, both(-kLog2e))));
    }
    return z;
}

template <int ACT>
__device__ __forceinline__ f32x2 act_slope2(f32x2 z)
{
    if constexpr (ACT == kRelu)
        return each(z, [](float x) { return x > 0.0f ? 1.0f : (x <= 0.0f ? 0.0f : x); });  // NaN stays NaN
    if constexpr (ACT == kGelu) {
        const f32x2 na = minus_abs14(z);
        const f32x2 u = mul2(gauss2(z), fma2(na, both(kInvSqrt2Pi), half_erfcx2(na)));
        float z0, z1, u0, u1, w0, w1;
        split(z, z0, z1);
        split(u, u0, u1);
        split(fma2(u, both(-1.0f), both(1.0f)), w0, w1);
        return pair(z0 < 0.0f ? u0 : w0, z1 < 0.0f ? u1 : w1);
    }
    if constexpr (ACT == kGeluTanh) {
        const f32x2 c = each(z, [](float x) { return max_nan(min_nan(x, 12.0f), -12.0f); });
        const f32x2 q = mul2(c, c);
        const f32x2 s = logistic2(mul2(c, fma2(q, both(-kTanhC1 * kLog2e), both(-kTanhC0 * kLog2e))));
        return fma2(mul2(mul2(c, s), fma2(s, both(-1.0f), both(1.0f))), fma2(q, both(3.0f * kTanhC1), both(kTanhC0)), s);
    }
    if constexpr (ACT == kSilu) {
        const f32x2 c = each(z, [](float x) { return max_nan(min_nan(x, 100.0f), -100.0f); });
        const f32x2 s = logistic2(mul2(c, both(-kLog2e)));
        return mul2(s, fma2(c, fma2(s, both(-1.0f), both(1.0f)), both(1.0f)));
    }
    return both(1.0f);
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
