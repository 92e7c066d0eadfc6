// Where column sums end: a vector of gradients.
#pragma once

#include "tile_kernel.cuh"

namespace dtg {
namespace linear {

// A bias gradient to be written: beta * dbias + sum, of type kOutF16, kOutBf16 or kOutF32.
struct BiasGrad {
    void* dbias;
    int32_t type;
    float beta;
};

__device__ __forceinline__ void write_bias_grad(const BiasGrad& b, int64_t n, float s)
{
    if (b.type == kOutF32) {
        float* d = static_cast<float*>(b.dbias) + n;
        *d = b.beta != 0.0f ? fmaf(b.beta, *d, s) : s;
    } else {
        uint16_t* d = static_cast<uint16_t*>(b.dbias) + n;
        const bool bf16 = b.type == kOutBf16;
        if (b.beta != 0.0f) s = fmaf(b.beta, bf16 ? load16<true>(d) : load16<false>(d), s);
        *d = bf16 ? cvt16<true>(__float_as_uint(s)) : cvt16<false>(__float_as_uint(s));
    }
}

}  // namespace linear
}  // namespace dtg
