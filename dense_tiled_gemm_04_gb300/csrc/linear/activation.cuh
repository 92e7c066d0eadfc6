// The activations of the linear-layer kernels and their derivatives, in fp32.
//
//   act        value                          slope
//   kRelu      z < 0 ? 0 : z                  z <= 0 ? 0 : 1
//   kGelu      z Phi(z)                       Phi(z) + z phi(z)
//   kGeluTanh  z s(2u)                        s + z s (1 - s) 2u',  2u = z (c0 + c1 z^2)
//   kSilu      z s(z)                         s (1 + z (1 - s))
// with Phi, phi the normal distribution and density and s the logistic function.
//
// z s(t) is computed as z / (1 + e^-t) with the fast exponential and division (a few ulp each,
// under the rounding to 16 bits by three decimal digits): 1 + tanh(u) would cancel for negative
// z, this form keeps its relative precision there.  Overflowing exponentials give the limit
// (z / inf = -0).  Slopes are computed at z clamped to a range outside which they equal their
// limits in fp32, so that no 0 * inf appears; the clamps are comparisons, which let NaN pass.
#pragma once

namespace dtg {
namespace linear {

constexpr int kActNone = 0, kRelu = 1, kGelu = 2, kGeluTanh = 3, kSilu = 4;  // gemm_act_t

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhC0 = 1.5957691216057308f;    // 2 sqrt(2/pi)
constexpr float kTanhC1 = 0.071354816272600249f;  // 2 sqrt(2/pi) 0.044715

__device__ __forceinline__ float clamp_nan(float z, float lim) { return z > lim ? lim : (z < -lim ? -lim : z); }

template <int ACT>
__device__ __forceinline__ float act_value(float z)
{
    if constexpr (ACT == kRelu) return z < 0.0f ? 0.0f : z;
    if constexpr (ACT == kGelu) return 0.5f * z * (1.0f + erff(z * kSqrtHalf));
    if constexpr (ACT == kGeluTanh) return __fdividef(z, 1.0f + __expf(-z * fmaf(kTanhC1 * z, z, kTanhC0)));
    if constexpr (ACT == kSilu) return __fdividef(z, 1.0f + __expf(-z));
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z)
{
    if constexpr (ACT == kRelu) return z <= 0.0f ? 0.0f : (z > 0.0f ? 1.0f : z);  // NaN stays NaN
    if constexpr (ACT == kGelu) {
        const float c = clamp_nan(z, 14.0f);
        return fmaf(c * kInvSqrt2Pi, __expf(-0.5f * c * c), fmaf(0.5f, erff(c * kSqrtHalf), 0.5f));
    }
    if constexpr (ACT == kGeluTanh) {
        const float c = clamp_nan(z, 12.0f);
        const float s = __fdividef(1.0f, 1.0f + __expf(-c * fmaf(kTanhC1 * c, c, kTanhC0)));
        return fmaf(c * s * (1.0f - s), fmaf(3.0f * kTanhC1 * c, c, kTanhC0), s);
    }
    if constexpr (ACT == kSilu) {
        const float c = clamp_nan(z, 100.0f);
        const float s = __fdividef(1.0f, 1.0f + __expf(-c));
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
