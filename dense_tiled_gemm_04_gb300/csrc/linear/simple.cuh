// Plain kernels of the linear-layer operators: one output element per thread, 32 x 32 tiles, fp32
// fused multiply-adds over the contraction.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "activation.cuh"
#include "gemm.h"

namespace dtg {
namespace linear {

__device__ __forceinline__ float load_as_float(const void* p, int64_t i, int dtype)
{
    switch (dtype) {
    case GEMM_DTYPE_F16: return __half2float(static_cast<const __half*>(p)[i]);
    case GEMM_DTYPE_BF16: return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    case GEMM_DTYPE_E4M3: return float(static_cast<const __nv_fp8_e4m3*>(p)[i]);
    case GEMM_DTYPE_E5M2: return float(static_cast<const __nv_fp8_e5m2*>(p)[i]);
    default: return static_cast<const float*>(p)[i];
    }
}

__device__ __forceinline__ void store_from_float(void* p, int64_t i, int dtype, float v)
{
    switch (dtype) {
    case GEMM_DTYPE_F16: static_cast<__half*>(p)[i] = __float2half_rn(v); break;
    case GEMM_DTYPE_BF16: static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v); break;
    default: static_cast<float*>(p)[i] = v; break;
    }
}

struct SimpleParams {
    const void* A;  // element (m, k) at A[m * a_m + k * a_k]
    const void* B;  // element (k, n) at B[k * b_k + n * b_n]
    void* C;
    const void* bias;
    const void* in;  // residual (forward) or pre-activations (backward)
    void* Z;
    float* partials;  // column sums of 32-row blocks
    int64_t M, N, K, a_m, a_k, b_k, b_n, ldc, ldin, ldz, pitch;
    int32_t dtype, out, bias_dtype, act, slope;  // slope: multiply by act'(in) instead of applying act
    float alpha, beta;
};

__global__ void simple_product_kernel(const SimpleParams p)
{
    __shared__ float a[32][33], b[32][33];
    const int tx = threadIdx.x, ty = threadIdx.y;
    const int64_t tiles_n = (p.N + 31) / 32;
    const int64_t m0 = blockIdx.x / tiles_n * 32, n0 = blockIdx.x % tiles_n * 32;
    const int64_t m = m0 + ty, n = n0 + tx;
    float acc = 0.0f;
    for (int64_t k0 = 0; k0 < p.K; k0 += 32) {
        a[ty][tx] = m < p.M && k0 + tx < p.K ? load_as_float(p.A, m * p.a_m + (k0 + tx) * p.a_k, p.dtype) : 0.0f;
        b[ty][tx] = k0 + ty < p.K && n < p.N ? load_as_float(p.B, (k0 + ty) * p.b_k + n * p.b_n, p.dtype) : 0.0f;
        __syncthreads();
        for (int k = 0; k < 32; ++k) acc = fmaf(a[ty][k], b[k][tx], acc);
        __syncthreads();
    }
    const bool inside = m < p.M && n < p.N;
    float v = p.alpha * acc;
    if (inside) {
        if (p.bias) v += load_as_float(p.bias, n, p.bias_dtype);
        if (p.Z) store_from_float(p.Z, m * p.ldz + n, p.out, v);
        if (p.slope) {
            const float z = p.in ? load_as_float(p.in, m * p.ldin + n, p.out) : 0.0f;
            DTG_ACT_SWITCH(p.act, v *= act_slope<ACT>(z));
        } else {
            DTG_ACT_SWITCH(p.act, v = act_value<ACT>(v));
            if (p.in) v += load_as_float(p.in, m * p.ldin + n, p.out);
        }
        if (p.beta != 0.0f) v = fmaf(p.beta, load_as_float(p.C, m * p.ldc + n, p.out), v);
        store_from_float(p.C, m * p.ldc + n, p.out, v);
    }
    if (p.partials) {
        a[ty][tx] = inside ? v : 0.0f;
        __syncthreads();
        if (ty == 0) {
            float s = 0.0f;
            for (int i = 0; i < 32; ++i) s += a[i][tx];
            if (n < p.N) p.partials[m0 / 32 * p.pitch + n] = s;
        }
    }
}

__global__ void simple_act_grad_kernel(const SimpleParams p)  // A: dY, in: Z, C: dZ (or null)
{
    __shared__ float d[32][33];
    const int tx = threadIdx.x, ty = threadIdx.y;
    const int64_t tiles_n = (p.N + 31) / 32;
    const int64_t m0 = blockIdx.x / tiles_n * 32, n0 = blockIdx.x % tiles_n * 32;
    const int64_t m = m0 + ty, n = n0 + tx;
    float v = 0.0f;
    if (m < p.M && n < p.N) {
        v = load_as_float(p.A, m * p.a_m + n, p.dtype);
        const float z = p.in ? load_as_float(p.in, m * p.ldin + n, p.dtype) : 0.0f;
        DTG_ACT_SWITCH(p.act, v *= act_slope<ACT>(z));
        if (p.C) store_from_float(p.C, m * p.ldc + n, p.dtype, v);
    }
    if (p.partials) {
        d[ty][tx] = v;
        __syncthreads();
        if (ty == 0) {
            float s = 0.0f;
            for (int i = 0; i < 32; ++i) s += d[i][tx];
            if (n < p.N) p.partials[m0 / 32 * p.pitch + n] = s;
        }
    }
}

// dbias[n] = beta * dbias[n] + the sum of `rows` partial sums of column n, in row order.
__global__ void simple_column_sum_kernel(const float* partials, int64_t rows, int64_t pitch, int64_t N, void* dbias,
                                         int32_t dtype, float beta)
{
    const int64_t n = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
    if (n >= N) return;
    float s = 0.0f;
    for (int64_t r = 0; r < rows; ++r) s += partials[r * pitch + n];
    if (beta != 0.0f) s = fmaf(beta, load_as_float(dbias, n, dtype), s);
    store_from_float(dbias, n, dtype, s);
}

}  // namespace linear
}  // namespace dtg
