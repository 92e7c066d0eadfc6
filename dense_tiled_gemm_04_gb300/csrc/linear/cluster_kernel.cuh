// The linear-layer products on few output tiles: one token, a batch of tokens, a small ragged layer.
//
// What bounds these calls is reading the weights once (one token through 4096 x 4096 bf16: 33.6 MB,
// 5 us at the measured copy rate) and, below that, latency; the persistent tile kernels leave most SMs without a tile
// there (20 us for that token).  So:
//  * The output's contiguous dimension ("features") takes the 128 rows of the MMA, the other ("tokens") its
//    N = 16, 32, 64 or 128 columns: one token costs 16 columns of padding, not 128 rows.
//        forward  features N from W (K-major),    tokens M from X (K-major)
//        dgrad    features K from W (M-major),    tokens M from dY (K-major)
//        wgrad    features K from X (M-major),    "tokens" N from dY (N-major)
//  * A tile's contraction is split over the CTAs of a cluster, up to 16, so that there are one or two CTAs per
//    SM even when there are 32 tiles.  Two fit per SM (under 113 KB of ring each), so their waits overlap.
//  * The partial sums meet through distributed shared memory: each CTA puts its 128 x BN block in its own shared memory
//    (the ring's, done with), and after a cluster barrier adds its share of the outputs over all ranks in rank
//    order -- no workspace, no atomics, the same result every time.  Adding in the same place the operator is
//    applied: four features of a token per thread, 8 or 16 bytes stored, bias and residual fetched before the barrier.
// Measured, cold L2, against the tile kernels: see the launch rule in linear_api.cu.
#pragma once

#include "tile_kernel.cuh"

namespace dtg {
namespace linear {

constexpr int kClusterThreads = 256;  // producer, MMA, four TMEM warps, two more for the joining
constexpr int kClusterTmemWarp0 = 2;
constexpr int kClusterMaxSplit = 16;

struct ClusterParams : KernelParams {  // M: tokens, N: features of the output; K: the contraction
    int32_t tiles_t;     // token tiles
    int32_t chunk_kb;    // K blocks per accumulator (at most kClusterAccs of them per CTA)
    int32_t act;
    const void* bias;
    int32_t bias_f32;
    const void* in;      // as in TileParams
    int64_t ldin;
    void* Z;
    int64_t ldz;
    float* partials;     // dgrad: a row of `pitch` column sums per token tile; null: none
    int64_t pitch;
};

// Accumulators of a CTA.  A chain of products on one accumulator is no longer than the tile kernels' chunks (see there); a
// longer share of K goes to further accumulators, which are added when they leave TMEM.  256 of its columns per CTA, as
// two CTAs share an SM.
template <int BN>
constexpr int kClusterAccs = 256 / BN;

template <int BN>
struct ClusterSmem {
    static constexpr int kStages = BN == 16 ? 6 : BN == 32 ? 5 : BN == 64 ? 4 : 3;
    static constexpr int kABytes = kBM * kRowBytes;
    static constexpr int kStageBytes = kABytes + BN * kRowBytes;
    static constexpr int kRing = kStages * kStageBytes;
    static constexpr int kSumBytes = BN * kBM * 4;   // the partial sums, [token][feature], in the ring's place
    static constexpr int kColOff = kRing;            // dgrad: column sums, kColRows rows of 128 floats
    static constexpr int kColRows = BN >= 64 ? kClusterThreads / 32 : 0;
    static constexpr int kBarOff = kColOff + kColRows * kBM * 4;
    static constexpr int kNumBars = 2 * kStages + 2;  // full, empty, accumulator full, drain
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;
    static constexpr int kAlloc = kMiscOff + 16 + 1024;
    static_assert(kSumBytes <= kRing, "the sums fit the ring");
    static_assert(kAlloc <= 113 * 1024, "two CTAs per SM");
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// N (16 or 32) columns of the warp's TMEM lanes from `taddr` on.
template <int N>
__device__ __forceinline__ void load_columns(uint32_t (&v)[32], uint32_t taddr)
{
    static_assert(N == 16 || N == 32, "columns of one load");
    if constexpr (N == 16)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
            "%14, %15}, [%16];"
            : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
              "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
            : "r"(taddr)
            : "memory");
    else
        ptx::tmem_ld_32x32b_x32(taddr, v);
    ptx::tmem_wait_ld();
}

// Four consecutive 16-bit values from column c of a row, as fp32 pairs; zeros from column n on.
template <bool BF16>
__device__ __forceinline__ void load4(f32x2 (&v)[2], const uint16_t* row, int32_t c, int32_t n)
{
    if (c + 4 <= n && (reinterpret_cast<uintptr_t>(row + c) & 7u) == 0) {
        const uint2 w = *reinterpret_cast<const uint2*>(row + c);
        v[0] = unpack2<BF16>(w.x);
        v[1] = unpack2<BF16>(w.y);
    } else {
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = c + e < n ? load16<BF16>(row + c + e) : 0.0f;
        v[0] = pair(f[0], f[1]);
        v[1] = pair(f[2], f[3]);
    }
}

__device__ __forceinline__ void load4f(f32x2 (&v)[2], const float* row, int32_t c, int32_t n)
{
    float f[4];
    if (c + 4 <= n && (reinterpret_cast<uintptr_t>(row + c) & 15u) == 0) {
        const float4 w = *reinterpret_cast<const float4*>(row + c);
        f[0] = w.x;
        f[1] = w.y;
        f[2] = w.z;
        f[3] = w.w;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = c + e < n ? row[c + e] : 0.0f;
    }
    v[0] = pair(f[0], f[1]);
    v[1] = pair(f[2], f[3]);
}

template <bool BF16>
__device__ __forceinline__ void store4(uint16_t* row, int32_t c, int32_t n, const f32x2 (&v)[2])
{
    const uint2 w = make_uint2(round2<BF16>(v[0]), round2<BF16>(v[1]));
    if (c + 4 <= n) {  // rows are multiples of 16 bytes apart, c a multiple of 4
        *reinterpret_cast<uint2*>(row + c) = w;
    } else {
        const uint32_t h[2] = {w.x, w.y};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + e < n) row[c + e] = static_cast<uint16_t>(h[e >> 1] >> ((e & 1) * 16));
    }
}

// IN, OUT, MODE as linear_tile_kernel; BN: tokens per tile.  The cluster's size is the launch's.
template <int BN, int IN, int OUT, int MODE>
__global__ void __launch_bounds__(kClusterThreads, 2)
    linear_cluster_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const ClusterParams p)
{
    using T = Operand<IN>;
    using L = ClusterSmem<BN>;
    constexpr int STAGES = L::kStages;
    constexpr bool AT = MODE != kForward;  // features' operand is M-major
    constexpr bool BT = MODE == kWgrad;    // tokens' operand is N-major
    constexpr bool kBf16 = OUT == kOutBf16;
    static_assert(!BT || BN % T::kNBlock == 0, "an N-major box is one 128-byte row");
    constexpr uint32_t kTmemCols = BN * kClusterAccs<BN>;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t* const smem = smem_raw + (base - raw_addr);
    const uint32_t bar0 = base + L::kBarOff;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    const uint32_t acc_bar = bar0 + 8u * (2 * STAGES), drain_bar = acc_bar + 8u;
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
    volatile int32_t* const abort_flag = reinterpret_cast<volatile int32_t*>(smem + L::kMiscOff + 4);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    uint32_t ranks;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
    const uint32_t rank = ptx::cluster_ctarank();
    const uint32_t tile = blockIdx.x / ranks;
    const int32_t tf = static_cast<int32_t>(tile / p.tiles_t), tt = static_cast<int32_t>(tile - tf * p.tiles_t);
    const int32_t f0 = tf * kBM, t0 = tt * BN;
    // This CTA's K blocks.
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.num_kb) * rank / ranks);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.num_kb) * (rank + 1) / ranks);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            ptx::mbar_init(empty_bar(s), 1);
        }
        ptx::mbar_init(acc_bar, 1);
        ptx::mbar_init(drain_bar, 1);
        *abort_flag = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&tmA);
        ptx::prefetch_tmap(&tmB);
    }
    __syncwarp();
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(ptx::smem_addr(tmem_slot), kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    Watchdog wd{abort_flag, &p};

    // This thread's share of the outputs: units of four features of a token, numbered token by token; this rank's are
    // [u0, u1), thread by thread.
    const int tokens = p.M - t0 < BN ? p.M - t0 : BN;
    const int units = tokens * (kBM / 4);
    const int u0 = static_cast<int>(static_cast<int64_t>(units) * rank / ranks);
    const int u1 = static_cast<int>(static_cast<int64_t>(units) * (rank + 1) / ranks);
    const int32_t f = f0 + 4 * ((u0 + static_cast<int>(threadIdx.x)) & 31);  // the features of all of its units (32 divides 256)
    // Residual, pre-activations or dW of one unit.
    auto fetch_in = [&](int u, f32x2 (&x)[2]) {
        x[0] = x[1] = 0;
        if (!p.in || f >= p.N) return;
        const int64_t t = t0 + (u >> 5);
        if constexpr (OUT == kOutF32)
            load4f(x, static_cast<const float*>(p.in) + t * p.ldin, f, p.N);
        else
            load4<kBf16>(x, static_cast<const uint16_t*>(p.in) + t * p.ldin, f, p.N);
    };

    if (warp == kProducerWarp) {
        if (lane == 0) {
            // ---------------------------------------------------------------- producer
            uint32_t armed_mask = 0, armed_parity = 0;
            int stage = 0;
            uint32_t phase = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!wd.wait(empty_bar(stage), phase ^ 1u, kRoleProducer, tile, kb)) break;
                // Test hook: the first CTA leaves its last stage unloaded and unarmed.
                if (!(p.fault_inject && blockIdx.x == 0 && kb == kb1 - 1)) {
                    const uint32_t sa = base + stage * L::kStageBytes, sb = sa + L::kABytes;
                    const int32_t k0 = kb * T::kStageK;
                    ptx::mbar_arrive_expect_tx(full_bar(stage), L::kStageBytes);
                    armed_mask |= 1u << stage;
                    armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
                    if constexpr (AT) {
#pragma unroll
                        for (int q = 0; q < kBM / T::kNBlock; ++q)
                            ptx::tma_load_2d(sa + q * (T::kStageK * 128), &tmA, f0 + q * T::kNBlock, k0, full_bar(stage));
                    } else {
                        ptx::tma_load_2d(sa, &tmA, k0, f0, full_bar(stage));
                    }
                    if constexpr (BT) {
#pragma unroll
                        for (int q = 0; q < BN / T::kNBlock; ++q)
                            ptx::tma_load_2d(sb + q * (T::kStageK * 128), &tmB, t0 + q * T::kNBlock, k0, full_bar(stage));
                    } else {
                        ptx::tma_load_2d(sb, &tmB, k0, t0, full_bar(stage));
                    }
                }
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            for (int s = 0; s < STAGES; ++s)  // no load outlives the ring
                if (armed_mask & (1u << s)) wd.drain(full_bar(s), (armed_parity >> s) & 1u);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            // ---------------------------------------------------------------- MMA issuer
            constexpr uint32_t idesc = idesc_mma<T::kFormat, BT, kBM, BN>() | (AT ? 1u << 15 : 0u);
            int stage = 0;
            uint32_t phase = 0;
            bool aborted = false;
            auto chunk = [&](int c0, int c1, uint32_t acc) {  // K blocks [c0, c1) on one accumulator
                for (int kb = c0; kb < c1; ++kb) {
                    if (!wd.wait(full_bar(stage), phase, kRoleMma, tile, kb)) {
                        aborted = true;
                        return;
                    }
                    ptx::tc_fence_after_sync();
                    const uint32_t sa = base + stage * L::kStageBytes, sb = sa + L::kABytes;
#pragma unroll
                    for (int k = 0; k < T::kStageK / T::kMmaK; ++k) {
                        const uint64_t adesc = AT ? smem_desc_sw128(sa + k * (T::kMmaK * 128), T::kStageK * 128, 1024)
                                                  : smem_desc_sw128(sa + k * 32, 16, 1024);
                        const uint64_t bdesc = BT ? smem_desc_sw128(sb + k * (T::kMmaK * 128), T::kStageK * 128, 1024)
                                                  : smem_desc_sw128(sb + k * 32, 16, 1024);
                        const uint32_t accumulate = (kb != c0 || k != 0) ? 1u : 0u;
                        if constexpr (T::kF8)
                            ptx::mma_f8_cta1(acc, adesc, bdesc, idesc, accumulate);
                        else
                            ptx::mma_f16_cta1(acc, adesc, bdesc, idesc, accumulate);
                    }
                    ptx::mma_commit_cta1(empty_bar(stage));
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            };
            // Mostly one chunk, in a loop of its own: a chunk's end as a condition in the K loop cost one token through
            // 4096 x 4096 0.17 us of 8.74, an outer loop over chunks alone 0.06, this 0.04.
            if (__builtin_expect(kb1 - kb0 <= p.chunk_kb, 1)) {
                chunk(kb0, kb1, tmem_base);
            } else {
                uint32_t acc = tmem_base;
                for (int c0 = kb0; c0 < kb1 && !aborted; c0 += p.chunk_kb, acc += BN)
                    chunk(c0, kb1 - c0 > p.chunk_kb ? c0 + p.chunk_kb : kb1, acc);
            }
            // The accumulator is complete -- or, after a wait that ran out, every MMA issued has finished.
            ptx::mma_commit_cta1(aborted ? drain_bar : acc_bar);
            if (aborted) wd.drain(drain_bar, 0);
        }
        __syncwarp();
    }

    // Every thread fetches what its first two units need beside the sums while the product runs.
    const int u = u0 + static_cast<int>(threadIdx.x);
    f32x2 bias[2] = {0, 0}, in0[2] = {0, 0}, in1[2] = {0, 0};
    if (MODE == kForward && p.bias && u < u1 && f < p.N) {
        if (p.bias_f32)
            load4f(bias, static_cast<const float*>(p.bias), f, p.N);
        else
            load4<kBf16>(bias, static_cast<const uint16_t*>(p.bias), f, p.N);
    }
    if (u < u1) fetch_in(u, in0);
    if (u + kClusterThreads < u1) fetch_in(u + kClusterThreads, in1);
    __syncwarp();  // the lanes' shares end at different units; TMEM loads and the cluster's barrier take whole warps

    if (warp >= kClusterTmemWarp0 && warp < kClusterTmemWarp0 + 4) {
        // ---------------------------------------------------------------- accumulator -> shared memory
        const int quad = warp & 3;
        const bool ok = __all_sync(0xFFFFFFFFu, kb0 == kb1 || wd.wait(acc_bar, 0, kRoleEpilogue, tile, -1));
        ptx::tc_fence_after_sync();
        // All loads and MMAs of this CTA are done: the ring is free.
        const uint32_t sum = base + 4u * (quad * 32 + lane);
        const uint32_t lanes = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
        constexpr int kStep = BN < 32 ? 16 : 32;
        auto leave = [&](int c, const uint32_t (&v)[32]) {
#pragma unroll
            for (int i = 0; i < kStep; ++i) st_shared_f32(sum + (c + i) * (kBM * 4), __uint_as_float(v[i]));
        };
        if (__builtin_expect(kb1 - kb0 <= p.chunk_kb, 1)) {
#pragma unroll
            for (int c = 0; c < BN; c += kStep) {
                uint32_t v[32];
                if (ok && kb0 < kb1 && c < tokens) {
                    load_columns<kStep>(v, lanes + c);
                    leave(c, v);
                } else if (c < tokens) {  // no K block of its own
#pragma unroll
                    for (int i = 0; i < kStep; ++i) v[i] = 0;
                    leave(c, v);
                }
            }
        } else if (ok) {
#pragma unroll 1
            for (int c = 0; c < tokens; c += kStep) {
                uint32_t v[32];
                load_columns<kStep>(v, lanes + c);
                for (int done = p.chunk_kb, a = 1; done < kb1 - kb0; done += p.chunk_kb, ++a) {
                    uint32_t w[32];
                    load_columns<kStep>(w, lanes + a * BN + c);
#pragma unroll
                    for (int i = 0; i < kStep; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(w[i]));
                }
                leave(c, v);
            }
        }
    }
    __syncwarp();
    ptx::tc_fence_before_sync();
    ptx::cluster_sync();  // every rank's sums are in its shared memory

    // ---------------------------------------------------------------- join, operator, store
    f32x2 col[2] = {0, 0};  // dgrad: sums of this thread's units
    // Unit i, whose sums are s.
    auto finish = [&](int i, f32x2 (&s)[2], const f32x2 (&in)[2]) {
        if (f >= p.N) return;
        const int64_t t = t0 + (i >> 5);
        const f32x2 alpha = both(p.alpha);
        if constexpr (MODE == kForward) {
            s[0] = fma2(alpha, s[0], bias[0]);
            s[1] = fma2(alpha, s[1], bias[1]);
            if (p.Z) store4<kBf16>(static_cast<uint16_t*>(p.Z) + t * p.ldz, f, p.N, s);
            DTG_ACT_SWITCH(p.act, {
                s[0] = act_value2<ACT>(s[0]);
                s[1] = act_value2<ACT>(s[1]);
            });
            if (p.in) {
                s[0] = add2(s[0], in[0]);
                s[1] = add2(s[1], in[1]);
            }
        } else if constexpr (MODE == kDgrad) {
            s[0] = mul2(alpha, s[0]);
            s[1] = mul2(alpha, s[1]);
            if (p.in) {
                DTG_ACT_SWITCH(p.act, {
                    s[0] = mul2(s[0], act_slope2<ACT>(in[0]));
                    s[1] = mul2(s[1], act_slope2<ACT>(in[1]));
                });
            }
            col[0] = add2(col[0], s[0]);
            col[1] = add2(col[1], s[1]);
        } else {
            s[0] = mul2(alpha, s[0]);
            s[1] = mul2(alpha, s[1]);
            if (p.in) {
                s[0] = fma2(both(p.beta), in[0], s[0]);
                s[1] = fma2(both(p.beta), in[1], s[1]);
            }
        }
        if constexpr (OUT == kOutF32) {
            float o[4];
            split(s[0], o[0], o[1]);
            split(s[1], o[2], o[3]);
            float* row = static_cast<float*>(p.C) + t * p.ldc;
            if (f + 4 <= p.N) {
                *reinterpret_cast<float4*>(row + f) = make_float4(o[0], o[1], o[2], o[3]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (f + e < p.N) row[f + e] = o[e];
            }
        } else {
            store4<kBf16>(static_cast<uint16_t*>(p.C) + t * p.ldc, f, p.N, s);
        }
    };
    if (*abort_flag == 0) {
        // Two units at a time, eight ranks' sums of each in flight, the inputs of the next two on their way.
        for (int i = u; i < u1; i += 2 * kClusterThreads) {
            const int j = i + kClusterThreads;
            f32x2 s0[2] = {0, 0}, s1[2] = {0, 0};
            for (uint32_t r0 = 0; r0 < ranks; r0 += 8) {
                float4 v[8], w[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r0 + r < ranks) {
                        const uint32_t at = ptx::mapa_shared(base, r0 + r);
                        v[r] = ld_cluster_f4(at + 16u * static_cast<uint32_t>(i));
                        if (j < u1) w[r] = ld_cluster_f4(at + 16u * static_cast<uint32_t>(j));
                    }
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r0 + r < ranks) {
                        s0[0] = add2(s0[0], pair(v[r].x, v[r].y));
                        s0[1] = add2(s0[1], pair(v[r].z, v[r].w));
                        if (j < u1) {
                            s1[0] = add2(s1[0], pair(w[r].x, w[r].y));
                            s1[1] = add2(s1[1], pair(w[r].z, w[r].w));
                        }
                    }
            }
            f32x2 next0[2] = {0, 0}, next1[2] = {0, 0};
            if (i + 2 * kClusterThreads < u1) fetch_in(i + 2 * kClusterThreads, next0);
            if (j + 2 * kClusterThreads < u1) fetch_in(j + 2 * kClusterThreads, next1);
            finish(i, s0, in0);
            if (j < u1) finish(j, s1, in1);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                in0[e] = next0[e];
                in1[e] = next1[e];
            }
        }
    }
    __syncwarp();
    if constexpr (MODE == kDgrad) {
        // Column sums of the tile: per thread over its units, then over the CTA's warps, then over the ranks, each in a
        // fixed order.
        float* const cols = reinterpret_cast<float*>(smem + L::kColOff);
        const int group = (u0 + static_cast<int>(threadIdx.x)) & 31;
        *reinterpret_cast<f32x2*>(&cols[warp * kBM + 4 * group]) = col[0];
        *reinterpret_cast<f32x2*>(&cols[warp * kBM + 4 * group + 2]) = col[1];
        __syncthreads();
        if (threadIdx.x < kBM) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < L::kColRows; ++w) s += cols[w * kBM + threadIdx.x];
            cols[threadIdx.x] = s;  // read above by this thread alone
        }
    }
    __syncwarp();
    ptx::cluster_sync();  // no rank's shared memory is read any more (dgrad: the sums of every rank are ready)
    if constexpr (MODE == kDgrad) {
        if (rank == 0 && p.partials && threadIdx.x < 32) {
            float4 s = ld_cluster_f4(base + L::kColOff + 16u * threadIdx.x);
            for (uint32_t r = 1; r < ranks; ++r) {
                const float4 v = ld_cluster_f4(ptx::mapa_shared(base, r) + L::kColOff + 16u * threadIdx.x);
                s.x += v.x;
                s.y += v.y;
                s.z += v.z;
                s.w += v.w;
            }
            float* row = p.partials + static_cast<int64_t>(tt) * p.pitch + f0;
            const float o[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (f0 + 4 * static_cast<int>(threadIdx.x) + e < p.N) row[4 * threadIdx.x + e] = o[e];
        }
        __syncwarp();
        ptx::cluster_sync();
    }
    if (warp == kMmaWarp) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem_base, kTmemCols);
    }
}

}  // namespace linear
}  // namespace dtg
