// Layer norm, forward and backward, and the rounding of matrices to 8 bits with block scales.  All are bound by memory: the
// kernels read their inputs once, keep them in registers, and write their outputs once, but for the layer norm of rows longer than
// registers hold (over 16384 columns forward, 8192 backward), which are read three times, and twice.
//
// Layer norm.  A row belongs to WARPS warps, CHUNKS times 8 elements (16 bytes) a lane, so statistics are taken in two passes
// over registers: the mean, then the mean square of x - mean, without the cancellation of E[x^2] - mean^2.
//   A block takes rows b, b + grid, ... and keeps the loads of the next ones in flight: every warp copies its own chunks of
// the rows ahead into its own places of a ring in shared memory (cp.async, 16 bytes a lane), which it alone reads, so the ring
// needs no barrier.  Of a warp's 256 columns lane l works on 4 l ... 4 l + 3 and 128 + 4 l ...: fp32 weights then are 16 bytes a
// lane side by side (with 8 columns a lane every load of them touched twice the lines, and L1 was 72 % busy).
//
// Backward, with x^ = (x - mean) rstd and g = dy w:
//   dx = rstd (g - mean(g) - x^ mean(g x^)) + residual,   dw = sum over rows of dy x^,   db = sum over rows of dy.
// A block takes rows b, b + grid, ...; every lane adds its columns' dw and db in registers over all of them, and writes
// one row of partial sums per block, which column_sum_kernel adds in a fixed order.
//
// Measured (one GB300, inputs larger than L2; the copy rate is 6.7 TB/s; bytes counted once each), over 64 to 128 M elements: forward
// 16384 x 8192 bf16 83 us (6.5 TB/s), from 256 to 16384 columns 5.1 to 6.5 TB/s, longer rows 2.5 to 2.7 (20480, 65536 columns);
// backward 16384 x 4096 with residual 85 us (6.3 TB/s), from 256 to 8192 columns with residual 5.8 to 6.8, longer rows 3.3 with and 2.3
// to 2.7 without; rows under 256 columns leave lanes idle: 128 columns 2.2 forward and 2.8 backward without residual, 64 1.1 and
// 1.4.  Quantization 8192 x 8192 33.4 us (6.0 TB/s), in 128 x 128 blocks 37.8; where the last strip of 256 columns is thin, 100000 x
// 520 44 us (3.5) and 260000 x 200 49 us (3.2).
//
// 8 bits.  For each block of 1 x 128 or 128 x 128 elements: s = max(a / F, 2^-126), a the largest magnitude, F the
// type's largest number; q = x r rounded to nearest even, r = 1 / s and x r rounded to fp32.  The bound on s keeps r finite.  A
// NaN or an infinity makes every value of its block stand for NaN (s is NaN; or s is infinite, r is 0 and finite values are 0).
#pragma once

#include "sums.cuh"

namespace dtg {
namespace linear {

constexpr int kNormWarps = 16;       // most warps of a block of the forward kernel, one block per SM
constexpr int kNormMaxStages = 3;    // most rows of a warp whose loads are in flight, forward
constexpr int kNormGradStages = 2;   // rows whose loads are in flight, backward
constexpr int kNormGradThreads = 512;  // of an SM, backward: 128 registers each
constexpr int64_t kNormMaxHeld = 16384, kNormGradMaxHeld = 8192;  // longest rows that are kept in registers

// A parameter vector of fp32 or of the matrices' 16-bit type, and how it can be read.
enum { kVecNone, kVecF32, kVec16, kVecF32Any, kVec16Any };  // absent; quads aligned to their size; any alignment
struct NormVector {
    const void* at;
    int32_t kind;
};

// Elements c ... c + 3 of a vector (c a multiple of 4) as fp32 pairs; `fill` where it is absent or past its n elements.
template <bool BF16>
__device__ __forceinline__ void load_vector4(f32x2* v, const NormVector& vec, int32_t c, int32_t n, float fill)
{
    if (vec.kind == kVecF32 && c + 4 <= n) {
        const float4 a = reinterpret_cast<const float4*>(vec.at)[c >> 2];
        v[0] = pair(a.x, a.y);
        v[1] = pair(a.z, a.w);
    } else if (vec.kind == kVec16 && c + 4 <= n) {
        const uint2 a = reinterpret_cast<const uint2*>(vec.at)[c >> 2];
        v[0] = unpack2<BF16>(a.x);
        v[1] = unpack2<BF16>(a.y);
    } else {
        float f[4] = {fill, fill, fill, fill};
        const bool f32 = vec.kind == kVecF32 || vec.kind == kVecF32Any;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (vec.kind != kVecNone && c + e < n)
                f[e] = f32 ? static_cast<const float*>(vec.at)[c + e] : load16<BF16>(static_cast<const uint16_t*>(vec.at) + c + e);
        v[0] = pair(f[0], f[1]);
        v[1] = pair(f[2], f[3]);
    }
}

// Elements [c, c + 8), likewise.
template <bool BF16>
__device__ __forceinline__ void load_vector8(f32x2 (&v)[4], const NormVector& vec, int64_t c, int64_t n, float fill)
{
    load_vector4<BF16>(v, vec, static_cast<int32_t>(c), static_cast<int32_t>(n), fill);
    load_vector4<BF16>(v + 2, vec, static_cast<int32_t>(c) + 4, static_cast<int32_t>(n), fill);
}

// Columns c ... c + 3 of a 16-bit row to memory, none from n on.
template <bool FULL>
__device__ __forceinline__ void store_row4(uint16_t* row, int32_t c, int32_t n, uint32_t w0, uint32_t w1)
{
    if constexpr (FULL) {
        *reinterpret_cast<uint2*>(row + c) = make_uint2(w0, w1);
    } else if (c + 4 <= n) {
        *reinterpret_cast<uint2*>(row + c) = make_uint2(w0, w1);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < n) row[c + e] = static_cast<uint16_t>((e < 2 ? w0 : w1) >> (16 * (e & 1)));
    }
}

__device__ __forceinline__ uint2 ld_shared_u2(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
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
template <bool FULL>
__device__ __forceinline__ void copy_row8(uint32_t to, const uint16_t* row, int32_t c, int32_t n)
{
    if constexpr (FULL) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(row + c) : "memory");
    } else {
        const int left = n - c, bytes = left >= 8 ? 16 : left > 0 ? 2 * left : 0;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(row + (left > 0 ? c : 0)), "r"(bytes) : "memory");
    }
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// All but the newest n groups, n < kNormMaxStages.
__device__ __forceinline__ void copies_wait(int n)
{
    static_assert(kNormMaxStages == 3, "a case for each");
    if (n == 0)
        copies_wait<0>();
    else if (n == 1)
        copies_wait<1>();
    else
        copies_wait<2>();
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

// The sum of a value (or of two) over the WARPS warps of a row, warps [group * WARPS, (group + 1) * WARPS) of the block, for
// all of their threads; they meet at a barrier of their own.  `shared` alternates between two
// places from call to call, so that one barrier a call keeps its writes apart from the reads of the call before.
template <int WARPS>
__device__ __forceinline__ float row_sum(float v, float* shared, int group)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    if constexpr (WARPS > 1) {
        shared += group * WARPS;
        if ((threadIdx.x & 31) == 0) shared[(threadIdx.x >> 5) % WARPS] = v;
        __syncwarp();
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(WARPS * 32) : "memory");
        if constexpr (WARPS == 2) {
            v = shared[0] + shared[1];
        } else {
            f32x2 s = 0;
#pragma unroll
            for (int w = 0; w < WARPS; w += 4) {
                const float4 f = *reinterpret_cast<const float4*>(shared + w);
                s = add2(s, add2(pair(f.x, f.y), pair(f.z, f.w)));
            }
            v = sum_of(s);
        }
    }
    return v;
}

template <int WARPS, bool ALONE>
__device__ __forceinline__ float2 row_sums(float2 v, float2* shared, int group)
{
    f32x2 s = pair(v.x, v.y);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s = add2(s, __shfl_xor_sync(0xFFFFFFFFu, s, off));
    if constexpr (WARPS > 1) {
        split(s, v.x, v.y);
        if constexpr (ALONE) {  // the block's only row
            if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
            __syncthreads();
        } else {
            shared += group * WARPS;
            if ((threadIdx.x & 31) == 0) shared[(threadIdx.x >> 5) % WARPS] = v;
            __syncwarp();
            asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(WARPS * 32) : "memory");
        }
        s = 0;
#pragma unroll
        for (int w = 0; w < WARPS; w += 2) {
            const float4 f = *reinterpret_cast<const float4*>(shared + w);
            s = add2(s, add2(pair(f.x, f.y), pair(f.z, f.w)));
        }
    }
    split(s, v.x, v.y);
    return v;
}

// s / n, corrected by what the product with 1 / n leaves: a quotient that fp32 holds comes out exact, so a row of one value
// has that mean, and no variance.  (An infinite quotient leaves inf - inf, NaN: it stands as it is.)
__device__ __forceinline__ float over(float s, float n, float inv_n)
{
    const float q = s * inv_n;
    return isinf(q) ? q : fmaf(fmaf(-q, n, s), inv_n, q);
}

struct NormParams {
    const uint16_t* X;
    uint16_t* Y;
    float *mean, *rstd;  // null: not kept
    NormVector w, b;
    int64_t M, N, ldx, ldy;
    float eps;
    int32_t stages;  // rows of a warp whose loads are in flight
};

__device__ __forceinline__ void st_shared_pairs(uint32_t addr, f32x2 a, f32x2 b)
{
    asm volatile("st.shared.v2.b64 [%0], {%1, %2};" ::"r"(addr), "l"(a), "l"(b) : "memory");
}

// Rows of a block's warps: `groups` of them at once, WARPS warps each.  The weights and biases are in shared memory as fp32: with
// the ring there L1 has little room, and read through it they came from L2 for every row.  FULL: rows are a multiple of 256.
// Dynamic shared memory: 8 bytes a column (rounded up to 256), then stages * CHUNKS * 512 bytes a warp.
template <bool BF16, int WARPS, int CHUNKS, bool FULL>
__global__ void __launch_bounds__(kNormWarps * 32, 1) layer_norm_kernel(const NormParams p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float shared[2][kNormWarps];
    const int32_t N = static_cast<int32_t>(p.N), pitch = (N + 255) & ~255;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int group = warp / WARPS, in_row = warp % WARPS;
    const uint32_t params = ptx::smem_addr(smem);  // weights, then biases
    const uint32_t ring = params + 8u * pitch + 512u * warp;
    auto place = [&](int stage, int k) { return ring + 512u * static_cast<uint32_t>((stage * CHUNKS + k) * warps); };
    auto first = [&](int k) { return (k * WARPS + in_row) * 256; };
    const int64_t step = gridDim.x * static_cast<int64_t>(warps / WARPS);
    int64_t row = blockIdx.x * static_cast<int64_t>(warps / WARPS) + group;
    auto fetch = [&](int stage, int64_t r) {
        if (r < p.M) {
            const uint16_t* const x = p.X + r * p.ldx;
#pragma unroll
            for (int k = 0; k < CHUNKS; ++k)
                if (first(k) < N) copy_row8<FULL>(place(stage, k) + 16u * lane, x, first(k) + 8 * lane, N);
        }
        copies_commit();
    };
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int stages = p.stages;
    for (int st = 0; st < stages; ++st) fetch(st, row + st * step);
    for (int32_t c = 4 * threadIdx.x; c < pitch; c += 4 * blockDim.x) {
        f32x2 w[2], b[2];
        load_vector4<BF16>(w, p.w, c, N, 1.0f);
        load_vector4<BF16>(b, p.b, c, N, 0.0f);
        st_shared_pairs(params + 4u * c, w[0], w[1]);
        st_shared_pairs(params + 4u * (pitch + c), b[0], b[1]);
    }
    __syncthreads();
    const float n = static_cast<float>(N), inv_n = 1.0f / n;
    int stage = 0;
    for (; row < p.M; row += step) {
        copies_wait(stages - 1);
        __syncwarp();
        f32x2 v[CHUNKS][4];
        f32x2 sum = 0;
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
            if (first(k) >= N) break;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const uint2 a = ld_shared_u2(place(stage, k) + 256u * q + 8u * lane);
                v[k][2 * q] = unpack2<BF16>(a.x);
                v[k][2 * q + 1] = unpack2<BF16>(a.y);
                sum = add2(sum, add2(v[k][2 * q], v[k][2 * q + 1]));
            }
        }
        const float mean = over(row_sum<WARPS>(sum_of(sum), shared[0], group), n, inv_n);
        // The sum has used what was in the warp's places.
        fetch(stage, row + stages * step);
        stage = stage + 1 == stages ? 0 : stage + 1;
        f32x2 sq = 0;
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
            if (first(k) >= N) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[k][i] = add2(v[k][i], both(-mean));
            if (!FULL && first(k) + 256 > N) {  // nothing past the row's end counts
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int32_t c = first(k) + 128 * (i >> 1) + 4 * lane + 2 * (i & 1);
                    float lo, hi;
                    split(v[k][i], lo, hi);
                    v[k][i] = pair(c < N ? lo : 0.0f, c + 1 < N ? hi : 0.0f);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) sq = fma2(v[k][i], v[k][i], sq);
        }
        const float rstd = rsqrtf(over(row_sum<WARPS>(sum_of(sq), shared[1], group), n, inv_n) + p.eps);
        if (lane == 0 && in_row == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
        uint16_t* const y = p.Y + row * p.ldy;
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
            if (first(k) >= N) break;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int32_t c = first(k) + 128 * q + 4 * lane;
                const float4 w = ld_shared_f4(params + 4u * c), b = ld_shared_f4(params + 4u * (pitch + c));
                const f32x2 lo = fma2(mul2(v[k][2 * q], both(rstd)), pair(w.x, w.y), pair(b.x, b.y));
                const f32x2 hi = fma2(mul2(v[k][2 * q + 1], both(rstd)), pair(w.z, w.w), pair(b.z, b.w));
                store_row4<FULL>(y, c, N, round2<BF16>(lo), round2<BF16>(hi));
            }
        }
    }
}

// A row of any length per block, read again (from L2) for each pass.
constexpr int kWideWarps = 16, kWideUnroll = 4;

template <bool BF16>
__global__ void __launch_bounds__(kWideWarps * 32, 2) layer_norm_wide_kernel(const NormParams p)
{
    __shared__ __align__(16) float shared[2][kWideWarps];
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    constexpr int64_t kStep = kWideWarps * 32 * int64_t(8);
    const int64_t row = blockIdx.x;
    const uint16_t* const x = p.X + row * p.ldx;
    // f(c, v) on every eight values from column c on, zeros past the row's end; kWideUnroll loads at once.
    auto pass = [&](auto f) {
        for (int64_t c0 = threadIdx.x * int64_t(8); c0 < p.N; c0 += kWideUnroll * kStep) {
            uint4 raw[kWideUnroll];
#pragma unroll
            for (int u = 0; u < kWideUnroll; ++u) raw[u] = load_row8(x, c0 + u * kStep, p.N);
#pragma unroll
            for (int u = 0; u < kWideUnroll; ++u) {
                f32x2 v[4];
                unpack8<BF16>(v, raw[u]);
                f(c0 + u * kStep, v);
            }
        }
    };
    f32x2 sum = 0;
    pass([&](int64_t, f32x2 (&v)[4]) { sum = add2(sum, add2(add2(v[0], v[1]), add2(v[2], v[3]))); });
    const float n = static_cast<float>(p.N), inv_n = 1.0f / n;
    const float mean = over(row_sum<kWideWarps>(sum_of(sum), shared[0], 0), n, inv_n);
    f32x2 sq = 0;
    pass([&](int64_t c, f32x2 (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f32x2 e = add2(v[i], both(-mean));
            if (c + 8 > p.N) {
                float lo, hi;
                split(e, lo, hi);
                e = pair(c + 2 * i < p.N ? lo : 0.0f, c + 2 * i + 1 < p.N ? hi : 0.0f);
            }
            sq = fma2(e, e, sq);
        }
    });
    const float rstd = rsqrtf(over(row_sum<kWideWarps>(sum_of(sq), shared[1], 0), n, inv_n) + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    pass([&](int64_t c, f32x2 (&v)[4]) {
        if (c >= p.N) return;
        f32x2 w[4], b[4];
        load_vector8<BF16>(w, p.w, c, p.N, 1.0f);
        load_vector8<BF16>(b, p.b, c, p.N, 0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = fma2(mul2(add2(v[i], both(-mean)), both(rstd)), w[i], b[i]);
        store_row8(p.Y + row * p.ldy, c, p.N, round8<BF16>(b));
    });
}

struct NormGradParams {
    const uint16_t *dY, *X, *residual;  // residual null: none
    const float *mean, *rstd;
    NormVector w;
    uint16_t* dX;
    float *dw, *db;    // partial sums: a row of `pitch` per block; null: not wanted
    // JOIN, few blocks: the last of them to finish adds the partial sums itself, in block order, and saves a launch.
    int32_t* arrived;  // zero before and after
    BiasGrad dw_out, db_out;
    float2* row_means;  // rows that registers do not hold: (mean(g), mean(g x^))
    int64_t M, N, lddy, ldx, ldr, lddx, pitch;
    int64_t block_rows;  // layer_norm_grad_wide_kernel: rows per block
};

// GROUPS rows of a block at once, WARPS warps each, whose sums are joined in shared memory at the end.  Dynamic shared memory:
// kNormGradStages * 3 * CHUNKS * 512 bytes a warp, for dy, x and the residual.  With e = x - mean the row's sums are those of g
// and (g rstd) e, and dx = rstd (g - mean(g) - e rstd mean(g rstd e)).  (Sums of g e leave fp32's range where rstd is 0; past a row's
// end, where g is 0, e rstd may.)
// JOIN: see NormGradParams (an instantiation of its own: with the joining's registers 16384 x 4096 took 94 us, without 89).
template <bool BF16, int WARPS, int CHUNKS, int GROUPS, bool FULL, bool JOIN>
__global__ void __launch_bounds__(WARPS * GROUPS * 32, kNormGradThreads / (WARPS * GROUPS * 32))
    layer_norm_grad_kernel(const NormGradParams p)
{
    static_assert(kNormGradStages == 2, "row_sums takes the stage for its place");
    constexpr int kWarps = WARPS * GROUPS;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float2 shared[2][kWarps];
    const int32_t N = static_cast<int32_t>(p.N);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = GROUPS == 1 ? 0 : warp / WARPS, in_row = GROUPS == 1 ? warp : warp % WARPS;
    const uint32_t ring = ptx::smem_addr(smem) + 512u * warp;
    auto place = [&](int stage, int which, int k) { return ring + 512u * static_cast<uint32_t>(((stage * 3 + which) * CHUNKS + k) * kWarps); };
    auto first = [&](int k) { return (k * WARPS + in_row) * 256; };
    const int64_t step = gridDim.x * static_cast<int64_t>(GROUPS);
    int64_t row = blockIdx.x * static_cast<int64_t>(GROUPS) + group;
    const bool has_res = p.residual != nullptr;
    auto fetch = [&](int stage, int64_t r) {
        if (r < p.M) {
#pragma unroll
            for (int k = 0; k < CHUNKS; ++k)
                if (first(k) < N) {
                    copy_row8<FULL>(place(stage, 0, k) + 16u * lane, p.dY + r * p.lddy, first(k) + 8 * lane, N);
                    copy_row8<FULL>(place(stage, 1, k) + 16u * lane, p.X + r * p.ldx, first(k) + 8 * lane, N);
                    if (has_res) copy_row8<FULL>(place(stage, 2, k) + 16u * lane, p.residual + r * p.ldr, first(k) + 8 * lane, N);
                }
        }
        copies_commit();
    };
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
#pragma unroll
    for (int st = 0; st < kNormGradStages; ++st) fetch(st, row + st * step);
    float mean = 0.0f, rstd = 0.0f, next_mean = 0.0f, next_rstd = 0.0f;
    auto fetch_stats = [&](int64_t r) {
        if (r < p.M) {
            next_mean = p.mean[r];
            next_rstd = p.rstd[r];
        }
    };
    fetch_stats(row);
    f32x2 w[CHUNKS][4];
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k)
#pragma unroll
        for (int q = 0; q < 2; ++q) load_vector4<BF16>(&w[k][2 * q], p.w, first(k) + 128 * q + 4 * lane, N, 1.0f);
    f32x2 dw[CHUNKS][4] = {}, db[CHUNKS][4] = {};
    const float n = static_cast<float>(N), inv_n = 1.0f / n;
    int stage = 0;
    auto take = [&](f32x2 (&v)[4], int which, int k) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint2 a = ld_shared_u2(place(stage, which, k) + 256u * q + 8u * lane);
            v[2 * q] = unpack2<BF16>(a.x);
            v[2 * q + 1] = unpack2<BF16>(a.y);
        }
    };
    for (; row < p.M; row += step) {
        mean = next_mean;
        rstd = next_rstd;
        fetch_stats(row + step);
        copies_wait<kNormGradStages - 1>();
        __syncwarp();
        f32x2 s1 = 0, s2 = 0;
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
            if (first(k) >= N) break;
            f32x2 dy[4], e[4];
            take(dy, 0, k);
            take(e, 1, k);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // Past the row's end dy is 0, so e counts nowhere.
                e[i] = add2(e[i], both(-mean));
                dw[k][i] = fma2(mul2(e[i], both(rstd)), dy[i], dw[k][i]);
                db[k][i] = add2(db[k][i], dy[i]);
                const f32x2 g = mul2(dy[i], w[k][i]);
                s1 = add2(s1, g);
                s2 = fma2(mul2(g, both(rstd)), e[i], s2);
            }
        }
        const float2 c = row_sums<WARPS, GROUPS == 1>(make_float2(sum_of(s1), sum_of(s2)), shared[stage], group);
        // g - mean(g) first, g rounded as for the mean (a mere product would be contracted with the subtraction): a row of one
        // column leaves exactly the residual.
        const f32x2 c1 = both(-over(c.x, n, inv_n)), c2 = both(-rstd * over(c.y, n, inv_n));
        uint16_t* const dx = p.dX + row * p.lddx;
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
            if (first(k) >= N) break;
            f32x2 d[4], e[4];
            take(d, 0, k);
            take(e, 1, k);
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = fma2(add2(e[i], both(-mean)), c2, add2(fma2(d[i], w[k][i], both(0.0f)), c1));
            if (has_res) {
                take(e, 2, k);
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = fma2(d[i], both(rstd), e[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = mul2(d[i], both(rstd));
            }
            store_row4<FULL>(dx, first(k) + 4 * lane, N, round2<BF16>(d[0]), round2<BF16>(d[1]));
            store_row4<FULL>(dx, first(k) + 128 + 4 * lane, N, round2<BF16>(d[2]), round2<BF16>(d[3]));
        }
        __syncwarp();  // the warp has used what was in its places
        fetch(stage, row + kNormGradStages * step);
        stage ^= 1;
    }
    if (!p.dw && !p.db) return;
    // This block's sums: the groups' added in shared memory, in the ring's place.  (The pitch is a multiple of 64.)
    auto put = [&](float* to, int32_t c, f32x2 lo, f32x2 hi) {
        float f[4];
        split(lo, f[0], f[1]);
        split(hi, f[2], f[3]);
        if (to && c < p.pitch) *reinterpret_cast<float4*>(to + blockIdx.x * p.pitch + c) = make_float4(f[0], f[1], f[2], f[3]);
    };
    if constexpr (GROUPS > 1) {
        constexpr int kQuads = WARPS * CHUNKS * 64;  // of a group's columns: (chunk, half, lane), a warp's side by side
        static_assert(GROUPS * kQuads * 16 <= kNormGradStages * 3 * CHUNKS * 512 * kWarps, "the sums of one vector fit the ring");
        f32x2* const parts = reinterpret_cast<f32x2*>(smem);
        copies_wait<0>();
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float* const to = which ? p.db : p.dw;
            __syncthreads();  // the ring, and the first vector's sums, are done with
#pragma unroll
            for (int k = 0; k < CHUNKS; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    parts[2 * (group * kQuads + (k * WARPS + in_row) * 64 + (i >> 1) * 32 + lane) + (i & 1)] = which ? db[k][i] : dw[k][i];
            __syncthreads();
            for (int e = threadIdx.x; e < kQuads; e += kWarps * 32) {
                f32x2 lo = 0, hi = 0;
#pragma unroll
                for (int r = 0; r < GROUPS; ++r) {
                    lo = add2(lo, parts[2 * (r * kQuads + e)]);
                    hi = add2(hi, parts[2 * (r * kQuads + e) + 1]);
                }
                put(to, (e >> 6) * 256 + 128 * ((e >> 5) & 1) + 4 * (e & 31), lo, hi);
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                put(p.dw, first(k) + 128 * q + 4 * lane, dw[k][2 * q], dw[k][2 * q + 1]);
                put(p.db, first(k) + 128 * q + 4 * lane, db[k][2 * q], db[k][2 * q + 1]);
            }
    }
    if constexpr (JOIN) {
        __shared__ bool last;
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) last = atomicAdd(p.arrived, 1) == static_cast<int>(gridDim.x) - 1;
        __syncthreads();
        if (!last) return;
        __threadfence();
        const int32_t quads = (N + 3) >> 2;
        for (int32_t i = threadIdx.x; i < 2 * quads; i += kWarps * 32) {
            const bool second = i >= quads;
            const int32_t c = 4 * (second ? i - quads : i);
            const float* from = second ? p.db : p.dw;
            if (!from) continue;
            float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
            for (unsigned b = 0; b < gridDim.x; ++b) {
                const float4 f = __ldcg(reinterpret_cast<const float4*>(from + b * p.pitch + c));
                s[0] += f.x;
                s[1] += f.y;
                s[2] += f.z;
                s[3] += f.w;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < N) write_bias_grad(second ? p.db_out : p.dw_out, c + e, s[e]);
        }
        if (threadIdx.x == 0) *p.arrived = 0;  // ready for the next launch
    }
}

// Rows that registers do not hold: first the means of every row, then dx and the sums by strips of columns.
constexpr int kMeansWarps = 8, kMeansUnroll = 4;

template <bool BF16>
__global__ void __launch_bounds__(kMeansWarps * 32, 4) layer_norm_grad_means_kernel(const NormGradParams p)
{
    __shared__ __align__(16) float2 shared[kMeansWarps];
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int64_t row = blockIdx.x;
    const float mean = p.mean[row], rstd = p.rstd[row];
    f32x2 s1 = 0, s2 = 0;
    constexpr int64_t kStep = kMeansWarps * 32 * int64_t(8);
    for (int64_t c0 = threadIdx.x * int64_t(8); c0 < p.N; c0 += kMeansUnroll * kStep) {
        uint4 dy[kMeansUnroll], x[kMeansUnroll];
#pragma unroll
        for (int u = 0; u < kMeansUnroll; ++u) {
            dy[u] = load_row8(p.dY + row * p.lddy, c0 + u * kStep, p.N);
            x[u] = load_row8(p.X + row * p.ldx, c0 + u * kStep, p.N);
        }
#pragma unroll
        for (int u = 0; u < kMeansUnroll; ++u) {
            if (c0 + u * kStep >= p.N) break;
            f32x2 g[4], h[4], w[4];
            unpack8<BF16>(g, dy[u]);
            unpack8<BF16>(h, x[u]);
            load_vector8<BF16>(w, p.w, c0 + u * kStep, p.N, 1.0f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                g[i] = mul2(g[i], w[i]);
                s1 = add2(s1, g[i]);
                // (Past the row's end g is 0, and (x - mean) rstd may be infinite.)
                s2 = fma2(mul2(g[i], both(rstd)), add2(h[i], both(-mean)), s2);
            }
        }
    }
    const float2 s = row_sums<kMeansWarps, true>(make_float2(sum_of(s1), sum_of(s2)), shared, 0);
    const float inv_n = 1.0f / static_cast<float>(p.N);
    if (threadIdx.x == 0) p.row_means[row] = make_float2(s.x * inv_n, s.y * inv_n);
}

// A block has 256 columns of block_rows rows, a warp every eighth of them, two at a time.
constexpr int kStripWarps = 8, kStripCols = 256, kStripRows = 2;

template <bool BF16>
__global__ void __launch_bounds__(kStripWarps * 32, 2) layer_norm_grad_wide_kernel(const NormGradParams p)
{
    __shared__ f32x2 parts[2][kStripWarps][kStripCols / 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = blockIdx.x * static_cast<int64_t>(kStripCols) + lane * 8;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    f32x2 w[4], dw[4] = {}, db[4] = {};
    load_vector8<BF16>(w, p.w, c, p.N, 1.0f);
    const int64_t r0 = blockIdx.y * p.block_rows, r1 = r0 + p.block_rows < p.M ? r0 + p.block_rows : p.M;
    const bool has_res = p.residual != nullptr;
    if (c < p.N)
        for (int64_t row0 = r0 + warp; row0 < r1; row0 += kStripRows * kStripWarps) {
            uint4 dy[kStripRows], x[kStripRows], res[kStripRows];
            float mean[kStripRows], rstd[kStripRows];
            float2 means[kStripRows];
#pragma unroll
            for (int u = 0; u < kStripRows; ++u) {
                const int64_t row = row0 + u * kStripWarps;
                if (row >= r1) break;
                dy[u] = load_row8(p.dY + row * p.lddy, c, p.N);
                x[u] = load_row8(p.X + row * p.ldx, c, p.N);
                res[u] = has_res ? load_row8(p.residual + row * p.ldr, c, p.N) : make_uint4(0, 0, 0, 0);
                mean[u] = p.mean[row];
                rstd[u] = p.rstd[row];
                means[u] = p.row_means[row];
            }
#pragma unroll
            for (int u = 0; u < kStripRows; ++u) {
                const int64_t row = row0 + u * kStripWarps;
                if (row >= r1) break;
                f32x2 g[4], h[4], d[4];
                unpack8<BF16>(g, dy[u]);
                unpack8<BF16>(h, x[u]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h[i] = mul2(add2(h[i], both(-mean[u])), both(rstd[u]));
                    dw[i] = fma2(g[i], h[i], dw[i]);
                    db[i] = add2(db[i], g[i]);
                    g[i] = mul2(g[i], w[i]);
                    d[i] = mul2(fma2(h[i], both(-means[u].y), add2(g[i], both(-means[u].x))), both(rstd[u]));
                }
                if (has_res) {
                    unpack8<BF16>(h, res[u]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) d[i] = add2(d[i], h[i]);
                }
                store_row8(p.dX + row * p.lddx, c, p.N, round8<BF16>(d));
            }
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
    // quantize_rows_kernel: strips of 256 columns; a block's next box is step_rows rows and step_strips strips on.
    int64_t step_rows;
    int32_t strips, step_strips;
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

// A scale for every 128 elements of a row: 16 lanes a block of them, two such blocks and kQuantRows rows a warp.  As many thread
// blocks as run at once take boxes of 32 rows by 256 columns in turn, along the rows first, with the next box's loads in flight
// (8192 x 8192: 33.5 us; a thread block for every box 38.6, for every 16 rows of four warps 37.0).
constexpr int kQuantWarps = 8, kQuantRows = 4, kQuantBlocks = 4;  // kQuantBlocks: of an SM

template <bool BF16, bool E5M2>
__global__ void __launch_bounds__(kQuantWarps * 32, kQuantBlocks) quantize_rows_kernel(const QuantizeParams p)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    uint4 ahead[kQuantRows];
    auto load = [&](int64_t r0, int64_t c) {
#pragma unroll
        for (int u = 0; u < kQuantRows; ++u) {
            const int64_t row = r0 + u * kQuantWarps + warp;
            ahead[u] = make_uint4(0, 0, 0, 0);
            if (row < p.M) ahead[u] = load_row8(p.X + row * p.ldx, c, p.K);
        }
    };
    // (The grid has no more blocks than there are boxes.)
    int32_t strip = static_cast<int32_t>(blockIdx.x % static_cast<uint32_t>(p.strips));
    int64_t next_r0 = blockIdx.x / static_cast<uint32_t>(p.strips) * int64_t(kQuantWarps * kQuantRows);
    int64_t next_c = strip * int64_t(256) + lane * 8;
    load(next_r0, next_c);
    while (next_r0 < p.M) {
        const int64_t r0 = next_r0, c = next_c;
        uint4 raw[kQuantRows];
        uint32_t largest[kQuantRows];
#pragma unroll
        for (int u = 0; u < kQuantRows; ++u) raw[u] = ahead[u];
        next_r0 += p.step_rows;
        if ((strip += p.step_strips) >= p.strips) {
            strip -= p.strips;
            next_r0 += kQuantWarps * kQuantRows;
        }
        next_c = strip * int64_t(256) + lane * 8;
        load(next_r0, next_c);
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
