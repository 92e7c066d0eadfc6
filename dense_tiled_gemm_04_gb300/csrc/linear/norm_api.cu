// Host side of gemm_run_layer_norm, gemm_run_layer_norm_grad and gemm_run_quantize: argument checks and launches.
#include <algorithm>
#include <cmath>

#include "api_common.cuh"
#include "norm.cuh"

using namespace dtg::host;
using namespace dtg::linear;

namespace {

void check_param(Checks& c, const void* at, gemm_dtype_t t, gemm_dtype_t matrix)
{
    if (!at) return;
    if (t != GEMM_DTYPE_F32 && t != matrix)
        c.add(GEMM_ERR_INVALID_ARG);
    else
        c.vector(at, t);
}

void check_stat(Checks& c, const float* at)
{
    c.vector(at, GEMM_DTYPE_F32);
}

NormVector vector_of(const void* at, gemm_dtype_t t)
{
    if (!at) return {nullptr, kVecNone};
    const bool f32 = t == GEMM_DTYPE_F32;
    if ((reinterpret_cast<uintptr_t>(at) & (f32 ? 15u : 7u)) != 0) return {at, f32 ? kVecF32Any : kVec16Any};
    return {at, f32 ? kVecF32 : kVec16};
}

unsigned blocks_for(int64_t rows, int64_t per_block) { return static_cast<unsigned>(cdiv(rows, per_block)); }

// A persistent kernel over rows.
template <class P>
gemm_status_t launch_rows(gemm_handle_t h, void (*fn)(P), int slot, int64_t blocks, int threads, int smem, int smem_max, const P& p, cudaStream_t s)
{
    if (!h->dev.attrs_set[kNormSlot0 + slot]) {
        if (cudaFuncSetAttribute(reinterpret_cast<const void*>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize, smem_max) != cudaSuccess)
            return GEMM_ERR_CUDA;
        h->dev.attrs_set[kNormSlot0 + slot] = true;
    }
    return launch_after(fn, static_cast<unsigned>(blocks), threads, static_cast<size_t>(smem), s, p);
}

// The shapes of the kernels for rows that registers hold, by steps of 256, 512, ... columns: warps and chunks of 8 elements a
// lane for a row; backward: rows a block.  Few warps with many chunks each spend less on the sums across warps and wait less at
// barriers; the backward kernel's sums of dw and db leave room for two chunks (with four its weights came from L2 for every row:
// 8192 x 8192 125 us).  Forward rows that fill eight warps of four chunks take those: 16384 x 8192 83 us, on four of eight 89; but
// 7168 columns 89 and 84, and what lies between is not measured; nor are eight warps of fewer chunks for shorter rows.
struct NormShape {
    int warps, chunks;
};
constexpr int kNormShapes = 8, kNormGradShapes = 6;
constexpr NormShape kShape[kNormShapes] = {{1, 1}, {1, 2}, {1, 4}, {1, 8}, {2, 8}, {4, 8}, {8, 8}, {8, 4}};
constexpr int kNormFilled = 7;  // its index
constexpr int kNormSmem = 229376;  // dynamic, beside the row sums
// Bytes of an SM's rows in flight that are enough: the fewest rows ahead that pass it, up to three, of a block with as many groups
// of warps as one can have (few rows have fewer, and are done before it matters).  More only spreads DRAM's reads among its
// writes (128 M elements in rows of 7168: one row 84 us, two 95; 8192 on eight warps of four chunks: one 98, two 83, four 87;
// 1000: one 95, two 85: any bound from 32769 to 57343 chooses the better of each).
constexpr int64_t kNormInFlight = 41500;
struct NormGradShape {
    int warps, chunks, groups;
    int threads() const { return 32 * warps * groups; }
};
constexpr NormGradShape kGradShape[kNormGradShapes] = {{1, 1, 8}, {1, 2, 8}, {2, 2, 4}, {4, 2, 2}, {8, 2, 1}, {16, 2, 1}};

int shape_for(int64_t N)
{
    int i = 0;
    for (int64_t n = 256; n < N; n *= 2) ++i;
    return i;
}

template <bool BF16, bool FULL, int I>
constexpr auto norm_fn()
{
    return &layer_norm_kernel<BF16, kShape[I].warps, kShape[I].chunks, FULL>;
}

template <bool BF16, bool FULL, bool JOIN, int I>
constexpr auto norm_grad_fn()
{
    return &layer_norm_grad_kernel<BF16, kGradShape[I].warps, kGradShape[I].chunks, kGradShape[I].groups, FULL, JOIN>;
}

template <bool BF16, bool FULL>
gemm_status_t launch_norm(gemm_handle_t h, const NormParams& q, cudaStream_t s)
{
    constexpr void (*kFn[kNormShapes])(const NormParams) = {norm_fn<BF16, FULL, 0>(), norm_fn<BF16, FULL, 1>(), norm_fn<BF16, FULL, 2>(),
                                                            norm_fn<BF16, FULL, 3>(), norm_fn<BF16, FULL, 4>(), norm_fn<BF16, FULL, 5>(),
                                                            norm_fn<BF16, FULL, 6>(), norm_fn<BF16, FULL, 7>()};
    NormParams p = q;
    const int i = p.N > 7680 && p.N <= 8192 ? kNormFilled : shape_for(p.N);
    const NormShape shape = kShape[i];
    // Few rows are spread over the SMs before a block takes several; eight warps at least bring in weights and biases.
    const int64_t most = kNormWarps / shape.warps, groups = std::min(most, std::max(cdiv(p.M, h->dev.num_sms), int64_t(8) / shape.warps));
    const int64_t blocks = std::min<int64_t>(cdiv(p.M, groups), h->dev.num_sms);
    const int64_t params = 8 * cdiv(p.N, 256) * 256, row = 512 * shape.chunks * shape.warps * groups;
    const int64_t wish = kNormInFlight / (most * 2 * p.N) + 1, fit = (kNormSmem - params) / row;
    p.stages = static_cast<int32_t>(std::min({wish, fit, int64_t(kNormMaxStages)}));
    return launch_rows<NormParams>(h, kFn[i], i + kNormShapes * (2 * FULL + BF16), blocks, static_cast<int>(32 * shape.warps * groups),
                                   static_cast<int>(params + p.stages * row), kNormSmem, p, s);
}

template <bool BF16>
gemm_status_t launch_norm(gemm_handle_t h, const NormParams& p, cudaStream_t s)
{
    if (p.N > kNormMaxHeld) return launch_after(&layer_norm_wide_kernel<BF16>, blocks_for(p.M, 1), kWideWarps * 32, 0, s, p);
    return p.N % 256 == 0 ? launch_norm<BF16, true>(h, p, s) : launch_norm<BF16, false>(h, p, s);
}

// Most rows of partial sums of dw and db: blocks that run at once on 152 SMs (fewer SMs: fewer; more: no more).
int64_t norm_grad_max_blocks(int64_t M, int64_t N)
{
    return std::min<int64_t>(M, N > 4096 && N <= kNormGradMaxHeld ? 152 : 304);
}

template <bool BF16, bool FULL>
gemm_status_t launch_norm_grad(gemm_handle_t h, const NormGradParams& q, int64_t* blocks, bool* summed, cudaStream_t s)
{
    constexpr void (*kFn[2][kNormGradShapes])(const NormGradParams) = {
        {norm_grad_fn<BF16, FULL, false, 0>(), norm_grad_fn<BF16, FULL, false, 1>(), norm_grad_fn<BF16, FULL, false, 2>(),
         norm_grad_fn<BF16, FULL, false, 3>(), norm_grad_fn<BF16, FULL, false, 4>(), norm_grad_fn<BF16, FULL, false, 5>()},
        {norm_grad_fn<BF16, FULL, true, 0>(), norm_grad_fn<BF16, FULL, true, 1>(), norm_grad_fn<BF16, FULL, true, 2>(),
         norm_grad_fn<BF16, FULL, true, 3>(), norm_grad_fn<BF16, FULL, true, 4>(), norm_grad_fn<BF16, FULL, true, 5>()}};
    const int i = shape_for(q.N);
    const NormGradShape shape = kGradShape[i];
    *blocks = std::min({cdiv(q.M, shape.groups), norm_grad_max_blocks(q.M, q.N), int64_t(h->dev.num_sms) * (kNormGradThreads / shape.threads())});
    // Up to 32 blocks the last one adds their sums (65 x 1000 fp16, 17 blocks: 8.7 us, 10.2 with a second launch, whose host part it
    // saves).  What that block reads grows with the row's length too, to 2 MB at 32 x 8192; those sizes are not measured.
    NormGradParams p = q;
    if (*blocks <= 32 && (p.dw || p.db)) {
        p.arrived = h->ws.counters + h->ws.counter_count;  // its own
        *summed = true;
    }
    const int smem = 3 * kNormGradStages * shape.chunks * 16 * shape.threads();
    return launch_rows<NormGradParams>(h, kFn[*summed][i], i + kNormShapes * (4 + 4 * *summed + 2 * FULL + BF16), *blocks, shape.threads(), smem, smem, p, s);
}

// summed: set where the kernel has written dw and db itself, not only `blocks` rows of partial sums.
template <bool BF16>
gemm_status_t launch_norm_grad(gemm_handle_t h, const NormGradParams& q, int64_t* blocks, bool* summed, cudaStream_t s)
{
    if (q.N <= kNormGradMaxHeld)
        return q.N % 256 == 0 ? launch_norm_grad<BF16, true>(h, q, blocks, summed, s) : launch_norm_grad<BF16, false>(h, q, blocks, summed, s);
    NormGradParams p = q;
    const gemm_status_t st = launch_after(&layer_norm_grad_means_kernel<BF16>, blocks_for(p.M, 1), kMeansWarps * 32, 0, s, p);
    if (st != GEMM_OK) return st;
    p.block_rows = cdiv(p.M, std::min(cdiv(p.M, 32), norm_grad_max_blocks(p.M, p.N)));
    *blocks = cdiv(p.M, p.block_rows);
    return launch_after(&layer_norm_grad_wide_kernel<BF16>, dim3(blocks_for(p.N, kStripCols), static_cast<unsigned>(*blocks)),
                        kStripWarps * 32, 0, s, p);
}

template <bool BF16, bool E5M2>
gemm_status_t launch_quantize(gemm_handle_t h, QuantizeParams& p, bool square, cudaStream_t s)
{
    if (square) {
        const dim3 grid(blocks_for(p.K, kScaleBlock), static_cast<unsigned>(std::min<int64_t>(cdiv(p.M, kScaleBlock), 65535)));
        return launch_after(&quantize_blocks_kernel<BF16, E5M2>, grid, 256, 0, s, p);
    }
    constexpr int64_t kRows = kQuantWarps * kQuantRows;
    const int64_t strips = cdiv(p.K, 256);
    int64_t blocks = std::min(strips * cdiv(p.M, kRows), int64_t(h->dev.num_sms) * kQuantBlocks);
    // One fewer where every block would keep its strip: a narrow last one is then taken by all in turn (65536 x 1000: 38 us, 47).
    if (strips > 1 && blocks > strips && blocks % strips == 0) --blocks;
    p.strips = static_cast<int32_t>(strips);
    p.step_strips = static_cast<int32_t>(blocks % strips);
    p.step_rows = blocks / strips * kRows;
    return launch_after(&quantize_rows_kernel<BF16, E5M2>, static_cast<unsigned>(blocks), kQuantWarps * 32, 0, s, p);
}

}  // namespace

extern "C" {

gemm_status_t gemm_run_layer_norm(gemm_handle_t h, const gemm_layer_norm_args_t* args, void* stream)
{
    if (!h || !args) return GEMM_ERR_INVALID_ARG;
    const gemm_layer_norm_args_t& a = *args;
    if (!is_16bit(a.dtype) || !std::isfinite(a.eps) || a.eps < 0.0f) return GEMM_ERR_INVALID_ARG;
    if (a.M < 0 || a.N < 0) return GEMM_ERR_INVALID_ARG;
    if (a.M == 0 || a.N == 0) return GEMM_OK;
    Checks c;
    if (a.M > kMaxDim || a.N > kMaxDim) c.add(GEMM_ERR_UNSUPPORTED);
    c.matrix(a.X, a.N, a.ldx, a.dtype);
    c.matrix(a.Y, a.N, a.ldy, a.dtype);
    check_param(c, a.weight, a.weight_dtype, a.dtype);
    check_param(c, a.bias, a.bias_dtype, a.dtype);
    check_stat(c, a.mean);
    check_stat(c, a.rstd);
    if (c.st != GEMM_OK) return c.st;
    DeviceGuard g(h->device);
    if (!g.ok) return GEMM_ERR_CUDA;
    NormParams p;
    p.X = static_cast<const uint16_t*>(a.X);
    p.Y = static_cast<uint16_t*>(a.Y);
    p.mean = a.mean;
    p.rstd = a.rstd;
    p.w = vector_of(a.weight, a.weight_dtype);
    p.b = vector_of(a.bias, a.bias_dtype);
    p.M = a.M;
    p.N = a.N;
    p.ldx = a.ldx;
    p.ldy = a.ldy;
    p.eps = a.eps;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return a.dtype == GEMM_DTYPE_BF16 ? launch_norm<true>(h, p, s) : launch_norm<false>(h, p, s);
}

int64_t gemm_layer_norm_grad_workspace_bytes(int64_t M, int64_t N)
{
    if (M <= 0 || N <= 0) return 0;
    return 8 * norm_grad_max_blocks(M, N) * sum_pitch(N) + (N > kNormGradMaxHeld ? 8 * M : 0);
}

gemm_status_t gemm_run_layer_norm_grad(gemm_handle_t h, const gemm_layer_norm_grad_args_t* args, void* stream)
{
    if (!h || !args) return GEMM_ERR_INVALID_ARG;
    const gemm_layer_norm_grad_args_t& a = *args;
    if (!is_16bit(a.dtype) || !std::isfinite(a.beta)) return GEMM_ERR_INVALID_ARG;
    if (a.M < 0 || a.N < 0) return GEMM_ERR_INVALID_ARG;
    if (a.N == 0) return GEMM_OK;
    Checks c;
    if (a.M > kMaxDim || a.N > kMaxDim) c.add(GEMM_ERR_UNSUPPORTED);
    check_param(c, a.weight, a.weight_dtype, a.dtype);
    check_param(c, a.dweight, a.dweight_dtype, a.dtype);
    check_param(c, a.dbias, a.dbias_dtype, a.dtype);
    const bool sums = a.dweight || a.dbias;
    if (a.M > 0) {
        c.matrix(a.dY, a.N, a.lddy, a.dtype);
        c.matrix(a.X, a.N, a.ldx, a.dtype);
        c.matrix(a.dX, a.N, a.lddx, a.dtype);
        if (a.residual) c.matrix(a.residual, a.N, a.ldr, a.dtype);
        if (!a.mean || !a.rstd) c.add(GEMM_ERR_INVALID_ARG);
        check_stat(c, a.mean);
        check_stat(c, a.rstd);
        const int64_t need = gemm_layer_norm_grad_workspace_bytes(a.M, a.N);
        if ((sums || a.N > kNormGradMaxHeld) && (a.workspace || need > GEMM_OWN_SUMS_BYTES)) {
            if (!a.workspace || a.workspace_bytes < need)
                c.add(GEMM_ERR_INVALID_ARG);
            else if ((reinterpret_cast<uintptr_t>(a.workspace) & 15u) != 0)
                c.add(GEMM_ERR_UNSUPPORTED);
        }
    }
    if (c.st != GEMM_OK) return c.st;
    DeviceGuard g(h->device);
    if (!g.ok) return GEMM_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    float* const partials = a.workspace ? static_cast<float*>(a.workspace) : h->sums;
    const int64_t pitch = sum_pitch(a.N), half = norm_grad_max_blocks(a.M, a.N) * pitch;
    const SumVector dw{a.dweight, a.dweight_dtype, a.beta}, db{a.dbias, a.dbias_dtype, a.beta};
    int64_t blocks = 0;
    bool summed = false;
    if (a.M > 0) {
        NormGradParams p = {};
        p.dY = static_cast<const uint16_t*>(a.dY);
        p.X = static_cast<const uint16_t*>(a.X);
        p.residual = static_cast<const uint16_t*>(a.residual);
        p.mean = a.mean;
        p.rstd = a.rstd;
        p.w = vector_of(a.weight, a.weight_dtype);
        p.dX = static_cast<uint16_t*>(a.dX);
        p.dw = a.dweight ? partials : nullptr;
        p.db = a.dbias ? partials + half : nullptr;
        p.row_means = reinterpret_cast<float2*>(partials + 2 * half);
        p.M = a.M;
        p.N = a.N;
        p.lddy = a.lddy;
        p.ldx = a.ldx;
        p.ldr = a.ldr;
        p.lddx = a.lddx;
        p.pitch = pitch;
        p.dw_out = bias_grad(dw);
        p.db_out = bias_grad(db);
        const gemm_status_t st = a.dtype == GEMM_DTYPE_BF16 ? launch_norm_grad<true>(h, p, &blocks, &summed, s)
                                                             : launch_norm_grad<false>(h, p, &blocks, &summed, s);
        if (st != GEMM_OK) return st;
    }
    return summed ? GEMM_OK : launch_sums(partials, blocks, a.N, dw, db, half, s);
}

gemm_status_t gemm_run_quantize(gemm_handle_t h, const gemm_quantize_args_t* args, void* stream)
{
    if (!h || !args) return GEMM_ERR_INVALID_ARG;
    const gemm_quantize_args_t& a = *args;
    if (!is_16bit(a.dtype) || !is_f8(a.q_dtype) || (a.block_rows != 1 && a.block_rows != kScaleBlock)) return GEMM_ERR_INVALID_ARG;
    if (a.M < 0 || a.K < 0) return GEMM_ERR_INVALID_ARG;
    if (a.M == 0 || a.K == 0) return GEMM_OK;
    Checks c;
    if (a.M > kMaxDim || a.K > kMaxDim) c.add(GEMM_ERR_UNSUPPORTED);
    c.matrix(a.X, a.K, a.ldx, a.dtype);
    c.matrix(a.Q, a.K, a.ldq, a.q_dtype);
    if (!a.scales || a.lds < cdiv(a.K, kScaleBlock)) c.add(GEMM_ERR_INVALID_ARG);
    c.vector(a.scales, GEMM_DTYPE_F32);
    if (c.st != GEMM_OK) return c.st;
    DeviceGuard g(h->device);
    if (!g.ok) return GEMM_ERR_CUDA;
    QuantizeParams p = {};
    p.X = static_cast<const uint16_t*>(a.X);
    p.Q = static_cast<uint8_t*>(a.Q);
    p.S = a.scales;
    p.M = a.M;
    p.K = a.K;
    p.ldx = a.ldx;
    p.ldq = a.ldq;
    p.lds = a.lds;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool square = a.block_rows != 1;
    if (a.dtype == GEMM_DTYPE_BF16)
        return a.q_dtype == GEMM_DTYPE_E5M2 ? launch_quantize<true, true>(h, p, square, s) : launch_quantize<true, false>(h, p, square, s);
    return a.q_dtype == GEMM_DTYPE_E5M2 ? launch_quantize<false, true>(h, p, square, s) : launch_quantize<false, false>(h, p, square, s);
}

}  // extern "C"
