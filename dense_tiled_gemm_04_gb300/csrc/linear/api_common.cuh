// What the host sides of the linear-layer entry points share: argument checks, and launches that overlap the stream's
// previous kernel.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "gemm.h"
#include "host/handle.cuh"
#include "sums.cuh"

namespace dtg {
namespace host {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 512;  // the edges of the last tiles still fit 32 bits
constexpr int64_t kScaleBlock = 128;  // elements that share a block scale
constexpr int64_t kSumRows = 32;   // rows of a partial column sum
constexpr int64_t kSumAlign = 64;  // its row pitch is a multiple of this many columns

inline bool is_16bit(gemm_dtype_t t) { return t == GEMM_DTYPE_F16 || t == GEMM_DTYPE_BF16; }
inline bool is_act(gemm_act_t a) { return a >= GEMM_ACT_NONE && a <= GEMM_ACT_SILU; }
inline int bytes_of(gemm_dtype_t t) { return t == GEMM_DTYPE_F32 ? 4 : elem_bytes(t); }

// A matrix argument of `cols` > 0 elements per row: null or too small a pitch is INVALID_ARG, a
// base or pitch that is not a multiple of 16 bytes UNSUPPORTED.
inline gemm_status_t check_matrix(const void* p, int64_t cols, int64_t ld, gemm_dtype_t t)
{
    if (!p || ld < cols) return GEMM_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0 || (ld & (16 / bytes_of(t) - 1)) != 0) return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

// INVALID_ARG outranks UNSUPPORTED, whatever the order of the arguments.
struct Checks {
    gemm_status_t st = GEMM_OK;
    void add(gemm_status_t s)
    {
        if (s == GEMM_ERR_INVALID_ARG || st == GEMM_OK) st = s;
    }
    void matrix(const void* p, int64_t cols, int64_t ld, gemm_dtype_t t) { add(check_matrix(p, cols, ld, t)); }
    void vector(const void* p, gemm_dtype_t t)
    {
        if ((reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(bytes_of(t) - 1)) != 0) add(GEMM_ERR_UNSUPPORTED);
    }
};

// Column sums: dbias's type and address, and the workspace for M x cols.
inline void check_sums(Checks& c, const void* dbias, gemm_dtype_t t, const void* ws, int64_t ws_bytes, int64_t M, int64_t cols)
{
    if (!dbias) return;
    c.vector(dbias, t);
    const int64_t need = gemm_bias_grad_workspace_bytes(M, cols);
    if (!ws && need <= GEMM_OWN_SUMS_BYTES) return;  // the handle's
    if (!ws || ws_bytes < need)
        c.add(GEMM_ERR_INVALID_ARG);
    else if ((reinterpret_cast<uintptr_t>(ws) & 15u) != 0)
        c.add(GEMM_ERR_UNSUPPORTED);
}

inline int64_t sum_pitch(int64_t cols) { return cdiv(cols, kSumAlign) * kSumAlign; }

// Kernels that start while the stream's previous kernel finishes (they wait for it themselves).
template <class... P, class... A>
gemm_status_t launch_after(void (*fn)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A... args)
{
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, static_cast<P>(args)...) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

// dbias[n] = beta * dbias[n] + the sum of `rows` rows of partial sums, whose pitch is sum_pitch(cols); a vector of `type`.
struct SumVector {
    void* to;
    gemm_dtype_t type;
    float beta;
};

inline linear::BiasGrad bias_grad(const SumVector& v)
{
    return {v.to, v.type == GEMM_DTYPE_F32 ? linear::kOutF32 : (v.type == GEMM_DTYPE_BF16 ? linear::kOutBf16 : linear::kOutF16), v.beta};
}

// One vector, or two (from `offset` floats on) in one launch; a null `to` is left out.
gemm_status_t launch_sums(const float* partials, int64_t rows, int64_t cols, const SumVector& first, const SumVector& second,
                          int64_t offset, cudaStream_t s);

}  // namespace host
}  // namespace dtg
