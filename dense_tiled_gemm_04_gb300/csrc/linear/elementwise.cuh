// The linear layer's kernels without a product: an activation's backward pass, and the column sums
// that it and the dgrad kernels share.  Both are bound by memory.
#pragma once

#include "tile_kernel.cuh"

namespace dtg {
namespace linear {

// dZ = dY * act'(Z) and its column sums over blocks of rows.
//
// Floor: 2 + 2 bytes read and 2 written per element.  A warp covers 256 columns of a row (16 bytes a lane), the
// eight warps of a block rows r, r + 8, ... of its block of rows, four of them in flight per warp.
// Each lane adds its eight columns in registers over all its rows; the eight warps' sums meet in shared memory in
// warp order, so a row of partial sums is written per block of rows (not per 32 rows).
constexpr int kActWarps = 8;
constexpr int kActCols = 256;   // columns per block
constexpr int kActUnroll = 4;   // rows in flight per warp

struct ActGradParams {
    const uint16_t* dY;
    const uint16_t* Z;   // null: act is none
    uint16_t* dZ;        // null: sums only
    float* partials;     // null: no sums; else a row of `pitch` columns per block of rows
    int64_t M, N, lddy, ldz, lddz, pitch;
    int64_t block_rows;  // rows per block, a multiple of kActWarps
};

__device__ __forceinline__ void load8(uint32_t (&r)[4], const uint16_t* row, int64_t col, int64_t N)
{
    uint4 v = make_uint4(0, 0, 0, 0);
    if (col + 8 <= N) {
        v = *reinterpret_cast<const uint4*>(row + col);
    } else if (col < N) {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (col + e < N) w[e >> 1] |= static_cast<uint32_t>(row[col + e]) << ((e & 1) * 16);
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    r[0] = v.x;
    r[1] = v.y;
    r[2] = v.z;
    r[3] = v.w;
}

template <bool BF16, int ACT>
__global__ void __launch_bounds__(kActWarps * 32, 3) act_grad_kernel(const ActGradParams p)
{
    __shared__ float sums[kActWarps][kActCols];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t col = blockIdx.x * static_cast<int64_t>(kActCols) + lane * 8;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    // Blocks of rows beyond the grid's second dimension are taken in turn.
    for (int64_t rb = blockIdx.y; rb * p.block_rows < p.M; rb += gridDim.y) {
        const int64_t r0 = rb * p.block_rows;
        const int64_t r1 = r0 + p.block_rows < p.M ? r0 + p.block_rows : p.M;
        float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int64_t r = r0 + warp; r < r1; r += kActWarps * kActUnroll) {
            uint32_t g[kActUnroll][4], z[kActUnroll][4];
#pragma unroll
            for (int u = 0; u < kActUnroll; ++u) {
                const int64_t row = r + u * kActWarps;
                const bool in = row < r1 && col < p.N;
                if (in) load8(g[u], p.dY + row * p.lddy, col, p.N);
                if (in && ACT != kActNone) load8(z[u], p.Z + row * p.ldz, col, p.N);
            }
#pragma unroll
            for (int u = 0; u < kActUnroll; ++u) {
                const int64_t row = r + u * kActWarps;
                if (row >= r1 || col >= p.N) continue;
                float d[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    d[2 * i] = unpack_lo<BF16>(g[u][i]);
                    d[2 * i + 1] = unpack_hi<BF16>(g[u][i]);
                    if constexpr (ACT != kActNone) {
                        d[2 * i] *= act_slope<ACT>(unpack_lo<BF16>(z[u][i]));
                        d[2 * i + 1] *= act_slope<ACT>(unpack_hi<BF16>(z[u][i]));
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] += d[i];
                if (p.dZ) {
                    uint32_t h[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) h[i] = pack2<BF16>(__float_as_uint(d[2 * i]), __float_as_uint(d[2 * i + 1]));
                    uint16_t* dst = p.dZ + row * p.lddz + col;
                    if (col + 8 <= p.N) {
                        *reinterpret_cast<uint4*>(dst) = make_uint4(h[0], h[1], h[2], h[3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (col + e < p.N) dst[e] = static_cast<uint16_t>(h[e >> 1] >> ((e & 1) * 16));
                    }
                }
            }
        }
        if (p.partials) {
            __syncthreads();  // the sums of the block of rows before have been read
#pragma unroll
            for (int i = 0; i < 8; ++i) sums[warp][lane * 8 + i] = acc[i];
            __syncthreads();
            const int64_t c = blockIdx.x * static_cast<int64_t>(kActCols) + threadIdx.x;
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kActWarps; ++w) s += sums[w][threadIdx.x];
            if (c < p.N) p.partials[rb * p.pitch + c] = s;
        }
    }
}

// dbias[n] = beta * dbias[n] + the sum over `rows` partial sums of column n.  32 columns a block; warp w adds rows
// w, w + 8, ..., and the eight warps' sums are added in warp order.
template <int DB>  // kOutF16, kOutBf16, kOutF32: type of dbias
__global__ void __launch_bounds__(256) column_sum_kernel(const float* partials, int64_t rows, int64_t pitch, int64_t N,
                                                         void* dbias, float beta)
{
    __shared__ float sums[8][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t n = blockIdx.x * int64_t(32) + lane;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    float s = 0.0f;
    if (n < N) {
#pragma unroll 8
        for (int64_t r = warp; r < rows; r += 8) s += partials[r * pitch + n];
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && n < N) {
#pragma unroll
        for (int w = 1; w < 8; ++w) s += sums[w][lane];
        if constexpr (DB == kOutF32) {
            float* d = static_cast<float*>(dbias) + n;
            *d = beta != 0.0f ? fmaf(beta, *d, s) : s;
        } else {
            uint16_t* d = static_cast<uint16_t*>(dbias) + n;
            if (beta != 0.0f) s = fmaf(beta, load16<DB == kOutBf16>(d), s);
            *d = cvt16<DB == kOutBf16>(__float_as_uint(s));
        }
    }
}

}  // namespace linear
}  // namespace dtg
