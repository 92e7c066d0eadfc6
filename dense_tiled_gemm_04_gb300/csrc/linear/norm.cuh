// Layer norm, forward and backward, and the rounding of matrices to 8 bits with block scales.  All are bound by memory: every
// kernel reads its inputs once, keeps them in registers, and writes its outputs once.
//
// Layer norm.  A row belongs to WARPS warps, CHUNKS times 8 elements (16 bytes) a lane, so statistics are taken in two passes
// over registers: the mean, then the mean square of x - mean, without the cancellation of E[x^2] - mean^2.  Rows of more
// elements than registers hold are read again for every pass.
//   A block takes rows b, b + grid, ... and keeps the loads of the next ones in flight: every lane copies its own chunks of
// the rows ahead into its own places of a ring in shared memory (cp.async), which it alone reads, so the ring needs no
// barrier.
//
// Backward, with x^ = (x - mean) rstd and g = dy w:
//   dx = rstd (g - mean(g) - x^ mean(g x^)) + residual,   dw = sum over rows of dy x^,   db = sum over rows of dy.
// A block takes rows b, b + grid, ...; every lane adds its columns' dw and db in registers over all of them, and writes
// one row of partial sums per block, which column_sum_kernel adds in a fixed order.
//
// 8 bits.  For each block of 1 x 128 or 128 x 128 elements: s = max(a / F, 2^-126), a the largest magnitude, F the
// type's largest number; q = x r rounded to nearest even, r = 1 / s and x r rounded to fp32.  The bound on s keeps r finite.  A
// NaN or an infinity makes every value of its block stand for NaN (s is NaN; or s is infinite, r is 0 and finite values are 0).
#pragma once

#include "tile_kernel.cuh"

namespace dtg {
namespace linear {

// Rows ahead whose loads are in flight, and blocks per SM (64 registers a thread; backward: 128).
constexpr int kNormStages = 3, kNormGradStages = 2;
constexpr int norm_blocks_per_sm(int threads) { return 1024 / threads; }
constexpr int norm_grad_blocks_per_sm(int threads) { return 512 / threads; }
constexpr int64_t kNormMaxHeld = 16384;  // longest row that is kept in registers

// A parameter or gradient vector of fp32 or of the matrices' 16-bit type; null: absent.
struct NormVector {
    const void* at;
    int32_t f32;
};

// Elements [c, c + 8) of a vector as fp32 pairs; `fill` where it is absent or past its n elements.
template <bool BF16>
__device__ __forceinline__ void load_vector8(f32x2 (&v)[4], const NormVector& vec, int64_t c, int64_t n, float fill)
{
    if (!vec.at || c >= n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = both(fill);
        return;
    }
    const int elem = vec.f32 ? 4 : 2;
    const uint8_t* at = static_cast<const uint8_t*>(vec.at) + c * elem;
    if (c + 8 <= n && (reinterpret_cast<uintptr_t>(at) & 15u) == 0) {
        if (vec.f32) {
            const float4 a = reinterpret_cast<const float4*>(at)[0], b = reinterpret_cast<const float4*>(at)[1];
            v[0] = pair(a.x, a.y);
            v[1] = pair(a.z, a.w);
            v[2] = pair(b.x, b.y);
            v[3] = pair(b.z, b.w);
        } else {
            const uint4 w = *reinterpret_cast<const uint4*>(at);
            v[0] = unpack2<BF16>(w.x);
            v[1] = unpack2<BF16>(w.y);
            v[2] = unpack2<BF16>(w.z);
            v[3] = unpack2<BF16>(w.w);
        }
        return;
    }
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        f[e] = c + e >= n ? fill
               : vec.f32  ? reinterpret_cast<const float*>(at)[e]
                          : load16<BF16>(reinterpret_cast<const uint16_t*>(at) + e);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pair(f[2 * i], f[2 * i + 1]);
}

// Elements [c, c + 8) of a 16-bit row (16-byte aligned at c), zeros from column n on.
__device__ __forceinline__ uint4 load_row8(const uint16_t* row, int64_t c, int64_t n)
{
    if (c + 8 <= n) return *reinterpret_cast<const uint4*>(row + c);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (c + e < n) w[e >> 1] |= static_cast<uint32_t>(row[c + e]) << (16 * (e & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store_row8(uint16_t* row, int64_t c, int64_t n, uint4 v)
{
    if (c + 8 <= n) {
        *reinterpret_cast<uint4*>(row + c) = v;
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (c + e < n) row[c + e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
}

// Start the copy of elements [c, c + 8) of a 16-bit row to 16 bytes of shared memory: zeros from column n on, which is not
// read.
__device__ __forceinline__ void copy_row8(uint32_t to, const uint16_t* row, int64_t c, int64_t n)
{
    const int64_t left = 2 * (n - c);
    const int bytes = left >= 16 ? 16 : left > 0 ? static_cast<int>(left) : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(row + (left > 0 ? c : 0)), "r"(bytes) : "memory");
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool BF16>
__device__ __forceinline__ void unpack8(f32x2 (&v)[4], uint4 w)
{
    v[0] = unpack2<BF16>(w.x);
    v[1] = unpack2<BF16>(w.y);
    v[2] = unpack2<BF16>(w.z);
    v[3] = unpack2<BF16>(w.w);
}

template <bool BF16>
__device__ __forceinline__ uint4 round8(const f32x2 (&v)[4])
{
    return make_uint4(round2<BF16>(v[0]), round2<BF16>(v[1]), round2<BF16>(v[2]), round2<BF16>(v[3]));
}

__device__ __forceinline__ float sum_of(f32x2 v)
{
    float lo, hi;
    split(v, lo, hi);
    return lo + hi;
}

// The sums of two values over the WARPS warps of a row, for all of their threads.  `parity` alternates between calls, so that
// one barrier a call keeps its writes apart from the reads of the call before.
template <int WARPS>
__device__ __forceinline__ float2 row_sums(float2 v, float2 (*shared)[WARPS], int parity)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, off);
        v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, off);
    }
    if constexpr (WARPS > 1) {
        if ((threadIdx.x & 31) == 0) shared[parity][threadIdx.x >> 5] = v;
        __syncthreads();
        v = shared[parity][0];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) {
            v.x += shared[parity][w].x;
            v.y += shared[parity][w].y;
        }
    }
    return v;
}

struct NormParams {
    const uint16_t* X;
    uint16_t* Y;
    float *mean, *rstd;  // null: not kept
    NormVector w, b;
    int64_t M, N, ldx, ldy;
    float eps;
};

// ROWS rows per block at once (more than one: WARPS is 1).  Dynamic shared memory: kNormStages * CHUNKS * 16 bytes a thread.
template <bool BF16, int WARPS, int CHUNKS, int ROWS>
__global__ void __launch_bounds__(WARPS * ROWS * 32, norm_blocks_per_sm(WARPS * ROWS * 32)) layer_norm_kernel(const NormParams p)
{
    static_assert(ROWS == 1 || WARPS == 1, "a block's barrier covers one row");
    constexpr int kThreads = WARPS * ROWS * 32;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float2 shared[2][WARPS];
    const int t = ROWS > 1 ? threadIdx.x & 31 : threadIdx.x;
    const uint32_t mine = ptx::smem_addr(ring) + 16u * threadIdx.x;
    auto slot = [&](int stage, int k) { return mine + 16u * kThreads * static_cast<uint32_t>(stage * CHUNKS + k); };
    auto column = [&](int k) { return (k * WARPS * 32 + t) * int64_t(8); };
    const int64_t step = gridDim.x * static_cast<int64_t>(ROWS);
    int64_t row = blockIdx.x * static_cast<int64_t>(ROWS) + (ROWS > 1 ? threadIdx.x >> 5 : 0);
    auto fetch = [&](int stage, int64_t r) {
        if (r < p.M) {
#pragma unroll
            for (int k = 0; k < CHUNKS; ++k) copy_row8(slot(stage, k), p.X + r * p.ldx, column(k), p.N);
        }
        copies_commit();
    };
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
#pragma unroll
    for (int st = 0; st < kNormStages; ++st) fetch(st, row + st * step);
    const float n = static_cast<float>(p.N);
    int stage = 0;
    for (; row < p.M; row += step) {
        copies_wait<kNormStages - 1>();
        f32x2 v[CHUNKS][4];
        f32x2 sum = 0;
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
            unpack8<BF16>(v[k], ld_shared_u4(slot(stage, k)));
            sum = add2(sum, add2(add2(v[k][0], v[k][1]), add2(v[k][2], v[k][3])));
        }
        // (Divided, not multiplied by 1 / n: a row of one value has exactly that mean, and no variance.)
        const float mean = row_sums<WARPS>(make_float2(sum_of(sum), 0.0f), shared, 0).x / n;
        // The sum has used what was in the slot.
        fetch(stage, row + kNormStages * step);
        stage = stage + 1 == kNormStages ? 0 : stage + 1;
        f32x2 sq = 0;
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
            const int64_t c = column(k);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[k][i] = add2(v[k][i], both(-mean));
            if (c + 8 > p.N) {  // nothing past the row's end counts
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float lo, hi;
                    split(v[k][i], lo, hi);
                    v[k][i] = pair(c + 2 * i < p.N ? lo : 0.0f, c + 2 * i + 1 < p.N ? hi : 0.0f);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) sq = fma2(v[k][i], v[k][i], sq);
        }
        const float rstd = 1.0f / sqrtf(row_sums<WARPS>(make_float2(sum_of(sq), 0.0f), shared, 1).x / n + p.eps);
        if (t == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
        uint16_t* const y = p.Y + row * p.ldy;
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
            const int64_t c = column(k);
            if (c >= p.N) break;
            f32x2 w[4], b[4];
            load_vector8<BF16>(w, p.w, c, p.N, 1.0f);
            load_vector8<BF16>(b, p.b, c, p.N, 0.0f);
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = fma2(mul2(v[k][i], both(rstd)), w[i], b[i]);
            store_row8(y, c, p.N, round8<BF16>(b));
        }
    }
}

constexpr int kWideWarps = 32;  // a row of any length per block, read again for each pass

template <bool BF16>
__global__ void __launch_bounds__(kWideWarps * 32) layer_norm_wide_kernel(const NormParams p)
{
    __shared__ float2 shared[2][kWideWarps];
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int64_t row = blockIdx.x, step = kWideWarps * 32 * int64_t(8);
    const uint16_t* const x = p.X + row * p.ldx;
    const int64_t c0 = threadIdx.x * int64_t(8);
    f32x2 v[4], sum = 0;
    for (int64_t c = c0; c < p.N; c += step) {
        unpack8<BF16>(v, load_row8(x, c, p.N));
        sum = add2(sum, add2(add2(v[0], v[1]), add2(v[2], v[3])));
    }
    const float n = static_cast<float>(p.N);
    const float mean = row_sums<kWideWarps>(make_float2(sum_of(sum), 0.0f), shared, 0).x / n;
    float sq = 0.0f;
    for (int64_t c = c0; c < p.N; c += step) {
        unpack8<BF16>(v, load_row8(x, c, p.N));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo, hi;
            split(add2(v[i], both(-mean)), lo, hi);
            if (c + 2 * i < p.N) sq = fmaf(lo, lo, sq);
            if (c + 2 * i + 1 < p.N) sq = fmaf(hi, hi, sq);
        }
    }
    const float rstd = 1.0f / sqrtf(row_sums<kWideWarps>(make_float2(sq, 0.0f), shared, 1).x / n + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    for (int64_t c = c0; c < p.N; c += step) {
        f32x2 w[4], b[4];
        unpack8<BF16>(v, load_row8(x, c, p.N));
        load_vector8<BF16>(w, p.w, c, p.N, 1.0f);
        load_vector8<BF16>(b, p.b, c, p.N, 0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = fma2(mul2(add2(v[i], both(-mean)), both(rstd)), w[i], b[i]);
        store_row8(p.Y + row * p.ldy, c, p.N, round8<BF16>(b));
    }
}

struct NormGradParams {
    const uint16_t *dY, *X, *residual;  // residual null: none
    const float *mean, *rstd;
    NormVector w;
    uint16_t* dX;
    float *dw, *db;    // partial sums: a row of `pitch` per block; null: not wanted
    float2* row_means;  // rows that registers do not hold: (mean(g), mean(g x^))
    int64_t M, N, lddy, ldx, ldr, lddx, pitch;
    int64_t block_rows;  // layer_norm_grad_wide_kernel: rows per block
};

// dx of eight elements from those of g (mean of g: c1, of g x^: c2), x^ and the residual.
template <bool BF16>
__device__ __forceinline__ uint4 norm_dx8(const f32x2 (&g)[4], const f32x2 (&h)[4], float2 c, float rstd, bool has_res, uint4 res)
{
    f32x2 d[4], r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = mul2(fma2(h[i], both(-c.y), add2(g[i], both(-c.x))), both(rstd));
    if (has_res) {
        unpack8<BF16>(r, res);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = add2(d[i], r[i]);
    }
    return round8<BF16>(d);
}

// ROWS rows of a block at once (more than one: WARPS is 1), joined in shared memory at the end.  Dynamic shared memory:
// kNormGradStages * 3 * CHUNKS * 16 bytes a thread, for dy, x and the residual.
template <bool BF16, int WARPS, int CHUNKS, int ROWS>
__global__ void __launch_bounds__(WARPS * ROWS * 32, norm_grad_blocks_per_sm(WARPS * ROWS * 32))
    layer_norm_grad_kernel(const NormGradParams p)
{
    static_assert(ROWS == 1 || WARPS == 1, "a block's barrier covers one row");
    static_assert(kNormGradStages == 2, "row_sums takes the stage for its parity");
    constexpr int kThreads = WARPS * ROWS * 32;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float2 shared[2][WARPS];
    const int t = ROWS > 1 ? threadIdx.x & 31 : threadIdx.x;
    const int group = ROWS > 1 ? threadIdx.x >> 5 : 0;
    const uint32_t mine = ptx::smem_addr(ring) + 16u * threadIdx.x;
    auto slot = [&](int stage, int which, int k) { return mine + 16u * kThreads * static_cast<uint32_t>((stage * 3 + which) * CHUNKS + k); };
    auto column = [&](int k) { return (k * WARPS * 32 + t) * int64_t(8); };
    const int64_t step = gridDim.x * static_cast<int64_t>(ROWS);
    int64_t row = blockIdx.x * static_cast<int64_t>(ROWS) + group;
    auto fetch = [&](int stage, int64_t r) {
        if (r < p.M) {
#pragma unroll
            for (int k = 0; k < CHUNKS; ++k) {
                copy_row8(slot(stage, 0, k), p.dY + r * p.lddy, column(k), p.N);
                copy_row8(slot(stage, 1, k), p.X + r * p.ldx, column(k), p.N);
                if (p.residual) copy_row8(slot(stage, 2, k), p.residual + r * p.ldr, column(k), p.N);
            }
        }
        copies_commit();
    };
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
#pragma unroll
    for (int st = 0; st < kNormGradStages; ++st) fetch(st, row + st * step);
    f32x2 dw[CHUNKS][4] = {}, db[CHUNKS][4] = {};
    const float inv_n = 1.0f / static_cast<float>(p.N);
    int stage = 0;
    for (; row < p.M; row += step) {
        const float mean = p.mean[row], rstd = p.rstd[row];
        copies_wait<kNormGradStages - 1>();
        f32x2 s1 = 0, s2 = 0;
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
            f32x2 g[4], h[4], w[4];
            unpack8<BF16>(g, ld_shared_u4(slot(stage, 0, k)));
            unpack8<BF16>(h, ld_shared_u4(slot(stage, 1, k)));
            load_vector8<BF16>(w, p.w, column(k), p.N, 1.0f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // Past the row's end dy is 0, so x^ counts nowhere.
                h[i] = mul2(add2(h[i], both(-mean)), both(rstd));
                dw[k][i] = fma2(g[i], h[i], dw[k][i]);
                db[k][i] = add2(db[k][i], g[i]);
                g[i] = mul2(g[i], w[i]);
                s1 = add2(s1, g[i]);
                s2 = fma2(g[i], h[i], s2);
            }
        }
        float2 c12 = row_sums<WARPS>(make_float2(sum_of(s1), sum_of(s2)), shared, stage & 1);
        c12.x *= inv_n;
        c12.y *= inv_n;
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
            const int64_t c = column(k);
            if (c >= p.N) break;
            f32x2 g[4], h[4], w[4];
            uint4 res = make_uint4(0, 0, 0, 0);
            if (p.residual) res = ld_shared_u4(slot(stage, 2, k));
            unpack8<BF16>(g, ld_shared_u4(slot(stage, 0, k)));
            unpack8<BF16>(h, ld_shared_u4(slot(stage, 1, k)));
            load_vector8<BF16>(w, p.w, c, p.N, 1.0f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[i] = mul2(add2(h[i], both(-mean)), both(rstd));
                g[i] = mul2(g[i], w[i]);
            }
            store_row8(p.dX + row * p.lddx, c, p.N, norm_dx8<BF16>(g, h, c12, rstd, p.residual != nullptr, res));
        }
        // The stores have used what was in the slots.
        fetch(stage, row + kNormGradStages * step);
        stage = stage + 1 == kNormGradStages ? 0 : stage + 1;
    }
    if (!p.dw && !p.db) return;
    // This block's sums: of its one row group, or of ROWS warps by way of shared memory.
    if constexpr (ROWS > 1) {
        __shared__ f32x2 parts[2][ROWS][CHUNKS * 32 * 4];
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                parts[0][group][(k * 32 + t) * 4 + i] = dw[k][i];
                parts[1][group][(k * 32 + t) * 4 + i] = db[k][i];
            }
        __syncthreads();
        for (int e = threadIdx.x; e < 2 * CHUNKS * 32 * 4; e += ROWS * 32) {
            const int which = e / (CHUNKS * 32 * 4), at = e % (CHUNKS * 32 * 4);
            f32x2 s = parts[which][0][at];
#pragma unroll
            for (int r = 1; r < ROWS; ++r) s = add2(s, parts[which][r][at]);
            float* const to = which ? p.db : p.dw;
            if (to && 2 * at < p.pitch) *reinterpret_cast<f32x2*>(to + blockIdx.x * p.pitch + 2 * at) = s;
        }
    } else {
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
            const int64_t c = (k * WARPS * 32 + t) * int64_t(8);
            if (c >= p.pitch) break;  // the pitch is a multiple of 64
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (p.dw) *reinterpret_cast<f32x2*>(p.dw + blockIdx.x * p.pitch + c + 2 * i) = dw[k][i];
                if (p.db) *reinterpret_cast<f32x2*>(p.db + blockIdx.x * p.pitch + c + 2 * i) = db[k][i];
            }
        }
    }
}

// Rows that registers do not hold: first the means of every row, then dx and the sums by strips of columns.
template <bool BF16>
__global__ void __launch_bounds__(kWideWarps * 32) layer_norm_grad_means_kernel(const NormGradParams p)
{
    __shared__ float2 shared[2][kWideWarps];
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int64_t row = blockIdx.x;
    const float mean = p.mean[row], rstd = p.rstd[row];
    f32x2 s1 = 0, s2 = 0;
    for (int64_t c = threadIdx.x * int64_t(8); c < p.N; c += kWideWarps * 32 * int64_t(8)) {
        f32x2 g[4], h[4], w[4];
        unpack8<BF16>(g, load_row8(p.dY + row * p.lddy, c, p.N));
        unpack8<BF16>(h, load_row8(p.X + row * p.ldx, c, p.N));
        load_vector8<BF16>(w, p.w, c, p.N, 1.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            g[i] = mul2(g[i], w[i]);
            s1 = add2(s1, g[i]);
            s2 = fma2(g[i], mul2(add2(h[i], both(-mean)), both(rstd)), s2);
        }
    }
    const float2 s = row_sums<kWideWarps>(make_float2(sum_of(s1), sum_of(s2)), shared, 0);
    const float inv_n = 1.0f / static_cast<float>(p.N);
    if (threadIdx.x == 0) p.row_means[row] = make_float2(s.x * inv_n, s.y * inv_n);
}

constexpr int kStripWarps = 8;
constexpr int kStripCols = 256;

template <bool BF16>
__global__ void __launch_bounds__(kStripWarps * 32) layer_norm_grad_wide_kernel(const NormGradParams p)
{
    __shared__ f32x2 parts[2][kStripWarps][kStripCols / 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = blockIdx.x * static_cast<int64_t>(kStripCols) + lane * 8;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    f32x2 w[4], dw[4] = {}, db[4] = {};
    load_vector8<BF16>(w, p.w, c, p.N, 1.0f);
    const int64_t r0 = blockIdx.y * p.block_rows, r1 = r0 + p.block_rows < p.M ? r0 + p.block_rows : p.M;
    if (c < p.N)
        for (int64_t row = r0 + warp; row < r1; row += kStripWarps) {
            const float mean = p.mean[row], rstd = p.rstd[row];
            f32x2 g[4], h[4];
            uint4 res = make_uint4(0, 0, 0, 0);
            unpack8<BF16>(g, load_row8(p.dY + row * p.lddy, c, p.N));
            unpack8<BF16>(h, load_row8(p.X + row * p.ldx, c, p.N));
            if (p.residual) res = load_row8(p.residual + row * p.ldr, c, p.N);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[i] = mul2(add2(h[i], both(-mean)), both(rstd));
                dw[i] = fma2(g[i], h[i], dw[i]);
                db[i] = add2(db[i], g[i]);
                g[i] = mul2(g[i], w[i]);
            }
            store_row8(p.dX + row * p.lddx, c, p.N, norm_dx8<BF16>(g, h, p.row_means[row], rstd, p.residual != nullptr, res));
        }
    if (!p.dw && !p.db) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        parts[0][warp][lane * 4 + i] = dw[i];
        parts[1][warp][lane * 4 + i] = db[i];
    }
    __syncthreads();
    const int which = threadIdx.x >> 7, at = threadIdx.x & 127;
    f32x2 s = parts[which][0][at];
#pragma unroll
    for (int r = 1; r < kStripWarps; ++r) s = add2(s, parts[which][r][at]);
    float* const to = which ? p.db : p.dw;
    const int64_t col = blockIdx.x * static_cast<int64_t>(kStripCols) + 2 * at;
    if (to && col < p.pitch) *reinterpret_cast<f32x2*>(to + blockIdx.y * p.pitch + col) = s;
}

// ---------------------------------------------------------------- 8 bits

struct QuantizeParams {
    const uint16_t* X;
    uint8_t* Q;
    float* S;
    int64_t M, K, ldx, ldq, lds;
};

constexpr int kScaleCols = 128;
constexpr float kMaxE4m3 = 448.0f, kMaxE5m2 = 57344.0f;

template <bool E5M2>
__device__ __forceinline__ uint32_t to_f8x2(f32x2 v)
{
    float lo, hi;
    split(v, lo, hi);
    uint16_t r;
    if constexpr (E5M2)
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Magnitudes of 16-bit floats order as their bits without the sign do, NaNs above infinity: the largest of two words' halves.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The largest magnitudes of eight values' even and odd ones.
__device__ __forceinline__ uint32_t largest8(uint4 raw)
{
    constexpr uint32_t kNoSigns = 0x7FFF7FFFu;
    return max_u16x2(max_u16x2(raw.x & kNoSigns, raw.y & kNoSigns), max_u16x2(raw.z & kNoSigns, raw.w & kNoSigns));
}

// The larger magnitude of a word's halves.
template <bool BF16>
__device__ __forceinline__ float larger_half(uint32_t w)
{
    f32x2 v = unpack2<BF16>(max_u16x2(w, w >> 16));
    float lo, hi;
    split(v, lo, hi);
    return lo;
}

template <bool E5M2>
__device__ __forceinline__ float scale_for(float largest)
{
    return max_nan(__fdiv_rn(largest, E5M2 ? kMaxE5m2 : kMaxE4m3), 1.1754943508222875e-38f);
}

template <bool BF16, bool E5M2>
__device__ __forceinline__ void store_f8x8(uint8_t* row, int64_t c, int64_t n, uint4 raw, float r)
{
    f32x2 v[4];
    unpack8<BF16>(v, raw);
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = to_f8x2<E5M2>(mul2(v[i], both(r)));
    const uint2 w = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
    if (c + 8 <= n) {
        *reinterpret_cast<uint2*>(row + c) = w;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < n) row[c + e] = static_cast<uint8_t>((e < 4 ? w.x : w.y) >> (8 * (e & 3)));
    }
}

// A scale for every 128 elements of a row: 16 lanes a block, two blocks and kQuantRows rows a warp.
constexpr int kQuantWarps = 8, kQuantRows = 4;

template <bool BF16, bool E5M2>
__global__ void __launch_bounds__(kQuantWarps * 32) quantize_rows_kernel(const QuantizeParams p)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = blockIdx.x * int64_t(256) + lane * 8;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    constexpr int64_t kBlockRows = kQuantWarps * kQuantRows;
    // Blocks of rows beyond the grid's second dimension are taken in turn.
    for (int64_t r0 = blockIdx.y * kBlockRows; r0 < p.M; r0 += gridDim.y * kBlockRows) {
        uint4 raw[kQuantRows];
        uint32_t largest[kQuantRows];
#pragma unroll
        for (int u = 0; u < kQuantRows; ++u) {
            const int64_t row = r0 + u * kQuantWarps + warp;
            raw[u] = make_uint4(0, 0, 0, 0);
            if (row < p.M) raw[u] = load_row8(p.X + row * p.ldx, c, p.K);
        }
#pragma unroll
        for (int u = 0; u < kQuantRows; ++u) {
            largest[u] = largest8(raw[u]);
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) largest[u] = max_u16x2(largest[u], __shfl_xor_sync(0xFFFFFFFFu, largest[u], off));
        }
        // Lane u of a block's 16 divides for row u: one division and one reciprocal for all rows.
        uint32_t own = largest[0];
#pragma unroll
        for (int u = 1; u < kQuantRows; ++u) own = (lane & 15) == u ? largest[u] : own;
        const float s = scale_for<E5M2>(larger_half<BF16>(own)), inverse = __frcp_rn(s);
        if ((lane & 15) < kQuantRows && (c - (lane & 15) * 8) < p.K) {
            const int64_t row = r0 + (lane & 15) * kQuantWarps + warp;
            if (row < p.M) p.S[row * p.lds + c / kScaleCols] = s;
        }
#pragma unroll
        for (int u = 0; u < kQuantRows; ++u) {
            const int64_t row = r0 + u * kQuantWarps + warp;
            const float r = __shfl_sync(0xFFFFFFFFu, inverse, (lane & 16) + u);
            if (row < p.M && c < p.K) store_f8x8<BF16, E5M2>(p.Q + row * p.ldq, c, p.K, raw[u], r);
        }
    }
}

// A scale for every 128 x 128 elements: a block of threads each, 8 rows of 8 elements a thread.
template <bool BF16, bool E5M2>
__global__ void __launch_bounds__(256) quantize_blocks_kernel(const QuantizeParams p)
{
    __shared__ uint32_t largest[8];
    const int64_t c = blockIdx.x * static_cast<int64_t>(kScaleCols) + (threadIdx.x & 15) * 8;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    for (int64_t rb = blockIdx.y; rb * kScaleCols < p.M; rb += gridDim.y) {
        const int64_t r0 = rb * kScaleCols + (threadIdx.x >> 4);
        uint4 raw[8];
        uint32_t a = 0;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            raw[u] = make_uint4(0, 0, 0, 0);
            if (r0 + 16 * u < p.M) raw[u] = load_row8(p.X + (r0 + 16 * u) * p.ldx, c, p.K);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) a = max_u16x2(a, largest8(raw[u]));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) a = max_u16x2(a, __shfl_xor_sync(0xFFFFFFFFu, a, off));
        __syncthreads();  // the block before has been read
        if ((threadIdx.x & 31) == 0) largest[threadIdx.x >> 5] = a;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 8; ++w) a = max_u16x2(a, largest[w]);
        const float s = scale_for<E5M2>(larger_half<BF16>(a)), r = __frcp_rn(s);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (r0 + 16 * u < p.M && c < p.K) store_f8x8<BF16, E5M2>(p.Q + (r0 + 16 * u) * p.ldq, c, p.K, raw[u], r);
        if (threadIdx.x == 0) p.S[rb * p.lds + blockIdx.x] = s;
    }
}

}  // namespace linear
}  // namespace dtg
