// Host side of the linear-layer entry points of include/gemm.h: argument checks and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "gemm.h"
#include "host/handle.cuh"
#include "simple.cuh"

using namespace dtg::host;

namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kSumRows = 32;   // rows of a partial column sum
constexpr int64_t kSumAlign = 64;  // its row pitch is a multiple of this many columns

bool is_16bit(gemm_dtype_t t) { return t == GEMM_DTYPE_F16 || t == GEMM_DTYPE_BF16; }
bool is_act(gemm_act_t a) { return a >= GEMM_ACT_NONE && a <= GEMM_ACT_SILU; }
int bytes_of(gemm_dtype_t t) { return t == GEMM_DTYPE_F32 ? 4 : elem_bytes(t); }

// A matrix argument of `cols` > 0 elements per row: null or too small a pitch is INVALID_ARG, a
// base or pitch that is not a multiple of 16 bytes UNSUPPORTED.
gemm_status_t check_matrix(const void* p, int64_t cols, int64_t ld, gemm_dtype_t t)
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
void check_sums(Checks& c, const void* dbias, gemm_dtype_t t, const void* ws, int64_t ws_bytes, int64_t M, int64_t cols)
{
    if (!dbias) return;
    c.vector(dbias, t);
    if (M == 0) return;
    if (!ws || ws_bytes < gemm_bias_grad_workspace_bytes(M, cols))
        c.add(GEMM_ERR_INVALID_ARG);
    else if ((reinterpret_cast<uintptr_t>(ws) & 15u) != 0)
        c.add(GEMM_ERR_UNSUPPORTED);
}

int64_t sum_pitch(int64_t cols) { return cdiv(cols, kSumAlign) * kSumAlign; }

gemm_status_t launched() { return cudaPeekAtLastError() == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA; }

gemm_status_t launch_product(const dtg::linear::SimpleParams& p, cudaStream_t s)
{
    dtg::linear::simple_product_kernel<<<static_cast<unsigned>(cdiv(p.M, 32) * cdiv(p.N, 32)), dim3(32, 32), 0, s>>>(p);
    return launched();
}

gemm_status_t launch_sums(const float* partials, int64_t M, int64_t cols, void* dbias, gemm_dtype_t t, float beta,
                          cudaStream_t s)
{
    dtg::linear::simple_column_sum_kernel<<<static_cast<unsigned>(cdiv(cols, 128)), 128, 0, s>>>(
        partials, cdiv(M, kSumRows), sum_pitch(cols), cols, dbias, t, beta);
    return launched();
}

}  // namespace

extern "C" {

int64_t gemm_bias_grad_workspace_bytes(int64_t M, int64_t cols)
{
    if (M <= 0 || cols <= 0) return 0;
    return 4 * cdiv(M, kSumRows) * sum_pitch(cols);
}

gemm_status_t gemm_run_linear(gemm_handle_t h, const gemm_linear_args_t* args, void* stream)
{
    if (!h || !args) return GEMM_ERR_INVALID_ARG;
    const gemm_linear_args_t& a = *args;
    if (!is_16bit(a.dtype) && !is_f8(a.dtype)) return GEMM_ERR_INVALID_ARG;
    if (!is_16bit(a.out_dtype) || (is_16bit(a.dtype) && a.out_dtype != a.dtype)) return GEMM_ERR_INVALID_ARG;
    if (!is_act(a.act) || !std::isfinite(a.alpha)) return GEMM_ERR_INVALID_ARG;
    if (a.M < 0 || a.N < 0 || a.K < 0) return GEMM_ERR_INVALID_ARG;
    if (a.bias && a.bias_dtype != GEMM_DTYPE_F32 && a.bias_dtype != a.out_dtype) return GEMM_ERR_INVALID_ARG;
    if (a.M == 0 || a.N == 0) return GEMM_OK;
    Checks c;
    if (a.M > kMaxDim || a.N > kMaxDim || a.K > kMaxDim) c.add(GEMM_ERR_UNSUPPORTED);
    if (a.K > 0) {
        c.matrix(a.X, a.K, a.ldx, a.dtype);
        c.matrix(a.W, a.K, a.ldw, a.dtype);
    }
    c.matrix(a.Y, a.N, a.ldy, a.out_dtype);
    if (a.bias) c.vector(a.bias, a.bias_dtype);
    if (a.residual) c.matrix(a.residual, a.N, a.ldr, a.out_dtype);
    if (a.Z) c.matrix(a.Z, a.N, a.ldz, a.out_dtype);
    if (c.st != GEMM_OK) return c.st;
    DeviceGuard g(h->device);
    if (!g.ok) return GEMM_ERR_CUDA;
    dtg::linear::SimpleParams p = {};
    p.A = a.X;
    p.B = a.W;
    p.C = a.Y;
    p.bias = a.bias;
    p.in = a.residual;
    p.Z = a.Z;
    p.M = a.M;
    p.N = a.N;
    p.K = a.K;
    p.a_m = a.ldx;
    p.a_k = 1;
    p.b_k = 1;
    p.b_n = a.ldw;
    p.ldc = a.ldy;
    p.ldin = a.ldr;
    p.ldz = a.ldz;
    p.dtype = a.dtype;
    p.out = a.out_dtype;
    p.bias_dtype = a.bias_dtype;
    p.act = a.act;
    p.alpha = a.alpha;
    return launch_product(p, static_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_run_linear_dgrad(gemm_handle_t h, const gemm_dgrad_args_t* args, void* stream)
{
    if (!h || !args) return GEMM_ERR_INVALID_ARG;
    const gemm_dgrad_args_t& a = *args;
    if (!is_16bit(a.dtype) || !is_act(a.act) || !std::isfinite(a.alpha) || !std::isfinite(a.beta_bias))
        return GEMM_ERR_INVALID_ARG;
    if (a.M < 0 || a.N < 0 || a.K < 0) return GEMM_ERR_INVALID_ARG;
    if (a.dbias && a.dbias_dtype != GEMM_DTYPE_F32 && a.dbias_dtype != a.dtype) return GEMM_ERR_INVALID_ARG;
    if (a.K == 0) return GEMM_OK;
    Checks c;
    if (a.M > kMaxDim || a.N > kMaxDim || a.K > kMaxDim) c.add(GEMM_ERR_UNSUPPORTED);
    if (a.M > 0) {
        if (a.N > 0) {
            c.matrix(a.dY, a.N, a.lddy, a.dtype);
            c.matrix(a.W, a.K, a.ldw, a.dtype);
        }
        if (a.act != GEMM_ACT_NONE) c.matrix(a.Z, a.K, a.ldz, a.dtype);
        c.matrix(a.dX, a.K, a.lddx, a.dtype);
    }
    check_sums(c, a.dbias, a.dbias_dtype, a.workspace, a.workspace_bytes, a.M, a.K);
    if (c.st != GEMM_OK) return c.st;
    DeviceGuard g(h->device);
    if (!g.ok) return GEMM_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a.M > 0) {
        dtg::linear::SimpleParams p = {};
        p.A = a.dY;
        p.B = a.W;
        p.C = a.dX;
        p.in = a.act != GEMM_ACT_NONE ? a.Z : nullptr;
        p.partials = a.dbias ? static_cast<float*>(a.workspace) : nullptr;
        p.pitch = sum_pitch(a.K);
        p.M = a.M;
        p.N = a.K;
        p.K = a.N;
        p.a_m = a.lddy;
        p.a_k = 1;
        p.b_k = a.ldw;
        p.b_n = 1;
        p.ldc = a.lddx;
        p.ldin = a.ldz;
        p.dtype = a.dtype;
        p.out = a.dtype;
        p.act = a.act;
        p.slope = 1;
        p.alpha = a.alpha;
        const gemm_status_t st = launch_product(p, s);
        if (st != GEMM_OK) return st;
    }
    if (!a.dbias) return GEMM_OK;
    return launch_sums(static_cast<const float*>(a.workspace), a.M, a.K, a.dbias, a.dbias_dtype, a.beta_bias, s);
}

gemm_status_t gemm_run_linear_wgrad(gemm_handle_t h, const gemm_wgrad_args_t* args, void* stream)
{
    if (!h || !args) return GEMM_ERR_INVALID_ARG;
    const gemm_wgrad_args_t& a = *args;
    if (!is_16bit(a.dtype) || (a.out_dtype != GEMM_DTYPE_F32 && a.out_dtype != a.dtype)) return GEMM_ERR_INVALID_ARG;
    if (!std::isfinite(a.alpha) || !std::isfinite(a.beta)) return GEMM_ERR_INVALID_ARG;
    if (a.M < 0 || a.N < 0 || a.K < 0) return GEMM_ERR_INVALID_ARG;
    if (a.N == 0 || a.K == 0) return GEMM_OK;
    Checks c;
    if (a.M > kMaxDim || a.N > kMaxDim || a.K > kMaxDim) c.add(GEMM_ERR_UNSUPPORTED);
    if (a.M > 0) {
        c.matrix(a.dY, a.N, a.lddy, a.dtype);
        c.matrix(a.X, a.K, a.ldx, a.dtype);
    }
    c.matrix(a.dW, a.K, a.lddw, a.out_dtype);
    if (c.st != GEMM_OK) return c.st;
    DeviceGuard g(h->device);
    if (!g.ok) return GEMM_ERR_CUDA;
    dtg::linear::SimpleParams p = {};
    p.A = a.dY;
    p.B = a.X;
    p.C = a.dW;
    p.M = a.N;
    p.N = a.K;
    p.K = a.M;
    p.a_m = 1;
    p.a_k = a.lddy;
    p.b_k = a.ldx;
    p.b_n = 1;
    p.ldc = a.lddw;
    p.dtype = a.dtype;
    p.out = a.out_dtype;
    p.alpha = a.alpha;
    p.beta = a.beta;
    return launch_product(p, static_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_run_act_grad(gemm_handle_t h, const gemm_act_grad_args_t* args, void* stream)
{
    if (!h || !args) return GEMM_ERR_INVALID_ARG;
    const gemm_act_grad_args_t& a = *args;
    if (!is_16bit(a.dtype) || !is_act(a.act) || !std::isfinite(a.beta_bias)) return GEMM_ERR_INVALID_ARG;
    if (a.M < 0 || a.N < 0) return GEMM_ERR_INVALID_ARG;
    if (a.dbias && a.dbias_dtype != GEMM_DTYPE_F32 && a.dbias_dtype != a.dtype) return GEMM_ERR_INVALID_ARG;
    if (a.N == 0) return GEMM_OK;
    Checks c;
    if (a.M > kMaxDim || a.N > kMaxDim) c.add(GEMM_ERR_UNSUPPORTED);
    if (a.M > 0) {
        c.matrix(a.dY, a.N, a.lddy, a.dtype);
        if (a.act != GEMM_ACT_NONE) c.matrix(a.Z, a.N, a.ldz, a.dtype);
        if (a.dZ) c.matrix(a.dZ, a.N, a.lddz, a.dtype);
    }
    check_sums(c, a.dbias, a.dbias_dtype, a.workspace, a.workspace_bytes, a.M, a.N);
    if (c.st != GEMM_OK) return c.st;
    DeviceGuard g(h->device);
    if (!g.ok) return GEMM_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a.M > 0 && (a.dZ || a.dbias)) {
        dtg::linear::SimpleParams p = {};
        p.A = a.dY;
        p.C = a.dZ;
        p.in = a.act != GEMM_ACT_NONE ? a.Z : nullptr;
        p.partials = a.dbias ? static_cast<float*>(a.workspace) : nullptr;
        p.pitch = sum_pitch(a.N);
        p.M = a.M;
        p.N = a.N;
        p.a_m = a.lddy;
        p.ldc = a.lddz;
        p.ldin = a.ldz;
        p.dtype = a.dtype;
        p.act = a.act;
        dtg::linear::simple_act_grad_kernel<<<static_cast<unsigned>(cdiv(a.M, 32) * cdiv(a.N, 32)), dim3(32, 32), 0, s>>>(p);
        const gemm_status_t st = launched();
        if (st != GEMM_OK) return st;
    }
    if (!a.dbias) return GEMM_OK;
    return launch_sums(static_cast<const float*>(a.workspace), a.M, a.N, a.dbias, a.dbias_dtype, a.beta_bias, s);
}

}  // extern "C"
