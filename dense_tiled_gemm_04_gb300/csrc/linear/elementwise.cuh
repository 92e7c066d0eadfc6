// The linear layer's kernels without a product: an activation's backward pass, and the column sums
// that it and the dgrad kernels share.  Both are bound by memory.
#pragma once

#include "sums.cuh"

namespace dtg {
namespace linear {

// dZ = dY * act'(Z) and its column sums over blocks of rows.
//
// Floor: 2 + 2 bytes read and 2 written per element.  A warp covers 256 columns of a row (16 bytes a lane), the
// eight warps of a block rows r, r + 8, ... of its block of rows, two of them in flight per warp and four blocks per SM
// (8192 x 8192 bf16 gelu with sums, when those took eight warps a block: 75.8 us; four rows and three blocks 82.0, one row
// and six blocks 86.0.  Now, with gelu_tanh: 69.5, 85 % of the copy rate).
// Each lane adds its eight columns in registers over all its rows; the eight warps' sums meet in shared memory in
// warp order, so a row of partial sums is written per block of rows (not per 32 rows).
constexpr int kActWarps = 8;
constexpr int kActCols = 256;   // columns per block
constexpr int kActUnroll = 2;   // rows in flight per warp

struct ActGradParams {
    const uint16_t* dY;
    const uint16_t* Z;   // null: act is none
    uint16_t* dZ;        // null: sums only
    float* partials;     // a row of `pitch` sums per block of rows; null: none, or one block of rows
    BiasGrad bias;       // one block of rows: its sums are the whole columns' (dbias null: no sums)
    int64_t M, N, lddy, ldz, lddz, pitch;
    int64_t block_rows;  // rows per block
};

// A warp's column sums in shared memory, written two at a time.
struct __align__(16) WarpSums {
    float col[kActCols];
};
static_assert(alignof(WarpSums) >= sizeof(f32x2), "pairs of sums are stored at once");

template <bool BF16, int ACT>
__global__ void __launch_bounds__(kActWarps * 32, 4) act_grad_kernel(const ActGradParams p)
{
    __shared__ WarpSums sums[kActWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t col = blockIdx.x * static_cast<int64_t>(kActCols) + lane * 8;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    // Blocks of rows beyond the grid's second dimension are taken in turn.
    for (int64_t rb = blockIdx.y; rb * p.block_rows < p.M; rb += gridDim.y) {
        const int64_t r0 = rb * p.block_rows;
        const int64_t left = p.M - r0;
        const int rows = static_cast<int>(left < p.block_rows ? left : p.block_rows);
        const uint16_t* g_at = p.dY + r0 * p.lddy + col;
        const uint16_t* z_at = ACT != kActNone ? p.Z + r0 * p.ldz + col : nullptr;
        uint16_t* d_at = p.dZ ? p.dZ + r0 * p.lddz + col : nullptr;
        f32x2 acc[4] = {0, 0, 0, 0};
        if (col + 8 <= p.N) {
            for (int r = warp; r < rows; r += kActWarps * kActUnroll) {
                uint4 g[kActUnroll], z[kActUnroll];
#pragma unroll
                for (int u = 0; u < kActUnroll; ++u) {
                    const int row = r + u * kActWarps;
                    if (row < rows) {
                        g[u] = *reinterpret_cast<const uint4*>(g_at + row * p.lddy);
                        if constexpr (ACT != kActNone) z[u] = *reinterpret_cast<const uint4*>(z_at + row * p.ldz);
                    }
                }
#pragma unroll
                for (int u = 0; u < kActUnroll; ++u) {
                    const int row = r + u * kActWarps;
                    if (row < rows) {
                        const uint32_t gw[4] = {g[u].x, g[u].y, g[u].z, g[u].w};
                        const uint32_t zw[4] = {z[u].x, z[u].y, z[u].z, z[u].w};
                        uint32_t h[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            f32x2 v = unpack2<BF16>(gw[i]);
                            if constexpr (ACT != kActNone) v = mul2(v, act_slope2<ACT>(unpack2<BF16>(zw[i])));
                            acc[i] = add2(acc[i], v);
                            h[i] = round2<BF16>(v);
                        }
                        if (d_at) *reinterpret_cast<uint4*>(d_at + row * p.lddz) = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                }
            }
        } else if (col < p.N) {  // the lane whose columns end inside its eight
            const int n = static_cast<int>(p.N - col);
            float tail[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            for (int r = warp; r < rows; r += kActWarps) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n) {
                        f32x2 v = unpack2<BF16>(g_at[r * p.lddy + e]);
                        if constexpr (ACT != kActNone) v = mul2(v, act_slope2<ACT>(unpack2<BF16>(z_at[r * p.ldz + e])));
                        float d, unused;
                        split(v, d, unused);
                        tail[e] += d;
                        if (d_at) d_at[r * p.lddz + e] = cvt16<BF16>(__float_as_uint(d));
                    }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = pair(tail[2 * i], tail[2 * i + 1]);
        }
        if (p.partials || p.bias.dbias) {
            __syncthreads();  // the sums of the block of rows before have been read
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<f32x2*>(&sums[warp].col[lane * 8 + 2 * i]) = acc[i];
            __syncthreads();
            const int64_t c = blockIdx.x * static_cast<int64_t>(kActCols) + threadIdx.x;
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kActWarps; ++w) s += sums[w].col[threadIdx.x];
            if (c < p.N) {
                if (p.partials)
                    p.partials[rb * p.pitch + c] = s;
                else
                    write_bias_grad(p.bias, c, s);
            }
        }
    }
}

// dbias[n] = beta * dbias[n] + the sum over `rows` partial sums of column n.  32 columns a block; warp w adds rows
// w, w + 16, ..., sixteen of them in flight, and the warps' sums are added in warp order.  Two vectors of one matrix of
// partial sums go in one launch: the grid's second row takes `second`, whose sums start `offset` floats on.
constexpr int kSumWarps = 16;

__global__ void __launch_bounds__(32 * kSumWarps) column_sum_kernel(const float* partials, int64_t rows, int64_t pitch,
                                                                    int64_t N, const BiasGrad first, const BiasGrad second,
                                                                    int64_t offset)
{
    __shared__ float sums[kSumWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t n = blockIdx.x * int64_t(32) + lane;
    const BiasGrad& b = blockIdx.y ? second : first;
    partials += blockIdx.y * offset;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    float s = 0.0f;
    if (n < N) {
#pragma unroll 16
        for (int64_t r = warp; r < rows; r += kSumWarps) s += partials[r * pitch + n];
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && n < N) {
#pragma unroll
        for (int w = 1; w < kSumWarps; ++w) s += sums[w][lane];
        write_bias_grad(b, n, s);
    }
}

}  // namespace linear
}  // namespace dtg
