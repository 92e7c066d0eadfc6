// The linear-layer products on tcgen05: persistent, warp-specialised tile kernels with the
// operator's arithmetic in the epilogue.
//
//   kForward  rows = tokens M, columns = outputs N, contraction K:   z = alpha X W^T + bias (kept on
//             request), Y = act(z) + residual.            X and W are K-major.
//   kDgrad    rows = tokens M, columns = inputs K, contraction N:    d = (alpha dY W) * act'(Z), dX = d,
//             and the sums of d over each warp's 32 rows.  dY is K-major, W N-major (its rows are the contraction).
//   kWgrad    rows = outputs N, columns = inputs K, contraction M:   dW = alpha dY^T X + beta dW.
//             Both operands have the contraction as rows: A is M-major, B N-major.
//
// The work schedule (tile raster, stream-K shares, backwards K walks, CTA pairs), the operand
// ring and the bounded waits are those of gemm_tcgen05_kernel.  What differs:
//
// Accumulation.  The tensor core's fp32 accumulator truncates: over one chain of 8192 products of
// N(0, 1) data it ends 9.5e-6 (relative, in norm) below the exact sum, 4.5e-6 over 4096, 2.9e-7 over
// 256, where fp32 fused multiply-adds stay at 1.6e-6 (8192).  So an item's K blocks run in chunks of
// chunk_kb; each chunk overwrites one of the two TMEM accumulators, and the epilogue warps
// add it to a running sum in their registers, rounding to nearest.  The MMAs of the next chunk
// run meanwhile, so the tensor pipe does not wait, and an item's accumulator is free as soon as its last
// chunk has been read, before any of the epilogue's arithmetic.  That is SUMS: where an fp32 result is wanted (weight
// gradients, column sums; chunks of 12 blocks), and contractions of more than 128 blocks.  A result that is rounded to 16
// bits alone takes a shorter contraction as one chunk, whose boxes go from TMEM straight through the epilogue.
//
// Epilogue.  Eight warps, two per TMEM lane quadrant, 32 rows x BN/2 columns each; with SUMS they hold
// those sums (128 registers at BN = 256; four warps would need 256 each).  Per box of 128 bytes of output
// columns: bias through the warp's staging buffer (every lane needs the same 64 values); the residual straight from
// global memory (16 bytes a load, a row's 128 bytes per lane, brought into L2 an item ahead) or, in dgrad, the
// pre-activations by TMA; then the 128-byte-swizzled staging buffer and a TMA store.
//
// What bounds it (one GB300, short bursts): 8192^3 bf16 forward with bias, gelu_tanh and z kept 577-588 us, as
// gemm_run's product alone (559-575).  16384 x 1024 x 8192: forward with residual 168-182 us (gemm_run 163-168), wgrad fp32
// accumulated 180-186 us; back to back, under the power limit, the three take 670-689, 197-203 and 189-193 us (gemm_run
// 8192^3 654-666).  dgrad of the tall layer with gelu takes 223 us, with sums 266 us (back to back 275-282), against 178
// without either: there a tile's MMAs (8192 cycles) leave the epilogue 32 issue slots an element, of which it takes 23, or
// 29 with the sums, at 0.4
// instructions a cycle -- two warps per scheduler waiting on fixed latencies, TMEM and shared memory.  Sixteen warps,
// loads a tile ahead, coalesced plain stores without the proxy fence, and rolled loops were slower.
//
// Column sums (kDgrad): the 32 lanes' rows are summed by five exchange steps that halve the columns
// a lane holds each time, which leaves two finished columns per lane and a fixed order of additions.
#pragma once

#include "activation.cuh"
#include "gemm_kernel.cuh"

namespace dtg {
namespace linear {

constexpr int kForward = 0, kDgrad = 1, kWgrad = 2;
constexpr int kOutF16 = 0, kOutBf16 = 1, kOutF32 = 2;
// Warps 0-3: producer, MMA and two idle ones; warps 4-11: epilogue.  setmaxnreg moves registers
// between them by warpgroup: the block starts with 384 x 168 = 64512, the first four warps go down
// to 64, the epilogue's eight up to 216 (128 x 64 + 256 x 216 = 63488).
constexpr int kTileThreads = 384;
constexpr int kTileLaunchRegs = 168;
constexpr int kTileMainRegs = 64;
constexpr int kTileEpiRegs = 216;
static_assert(128 * kTileMainRegs + 256 * kTileEpiRegs <= kTileThreads * kTileLaunchRegs, "the pool covers both shares");
constexpr int kTileEpiWarp0 = 4;
constexpr int kTileEpiWarps = 8;
constexpr int kTileStgBytes = 4096;   // one warp's 32 rows x 128 bytes
constexpr int kTileEpiBarrier = 1;

struct TileParams : KernelParams {
    int32_t chunk_kb;     // K blocks accumulated in TMEM before they join the fp32 registers' sums
    int32_t act;          // gemm_act_t
    const void* bias;     // forward; null: none
    int32_t bias_f32;     // bias is fp32 (else of the output type)
    const void* in;       // forward: residual; dgrad: pre-activations; wgrad: dW when beta != 0; null: none
    int64_t ldin;
    void* Z;              // forward: where z is kept; null: nowhere
    int64_t ldz;
    float* partials;      // dgrad: sums of 32-row blocks, `pitch` columns a row; null: none
    int64_t pitch;
};

// STG_BUFS: staging buffers per epilogue warp.
template <int B_ROWS, int STAGES, int STG_BUFS>
struct TileSmem {
    static constexpr int kABytes = kBM * kRowBytes;
    static constexpr int kStageBytes = kABytes + B_ROWS * kRowBytes;
    static constexpr int kStgOff = STAGES * kStageBytes;
    static constexpr int kStgBufs = STG_BUFS;
    static constexpr int kBarOff = kStgOff + kTileEpiWarps * STG_BUFS * kTileStgBytes;
    // full, empty, acc_full[2], acc_empty[2], drain, pre-activation boxes per staging buffer
    static constexpr int kNumBars = 2 * STAGES + 5 + kTileEpiWarps * 2;
    static constexpr int kMiscOff = kBarOff + kNumBars * 8;
    static constexpr int kTotal = kMiscOff + 16;  // tmem slot, abort flag, stream-K "last" flag
    static constexpr int kAlloc = kTotal + 1024;  // slack for aligning the base to 1 KB
    static_assert(kStageBytes % 1024 == 0 && kStgOff % 1024 == 0, "swizzle atoms need 1 KB alignment");
    static_assert(kAlloc <= 227 * 1024, "fits an SM");
};

template <int N>
__device__ __forceinline__ void registers_down()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int N>
__device__ __forceinline__ void registers_up()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Barriers, TMEM loads and cluster barriers are .aligned: a warp's threads execute them together, so code that its
// lanes leave at different points ends in __syncwarp() before one of them.
__device__ __forceinline__ void tile_epi_sync()
{
    __syncwarp();
    asm volatile("bar.sync %0, %1;" ::"n"(kTileEpiBarrier), "n"(kTileEpiWarps * 32) : "memory");
}

// Barrier of the eight epilogue warps that also ANDs a flag over their threads.
__device__ __forceinline__ bool tile_epi_and(bool v)
{
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred pi, po;\n\t"
        "setp.ne.u32 pi, %1, 0;\n\t"
        "bar.red.and.pred po, %2, %3, pi;\n\t"
        "selp.u32 %0, 1, 0, po;\n\t}\n"
        : "=r"(r)
        : "r"(v ? 1u : 0u), "n"(kTileEpiBarrier), "n"(kTileEpiWarps * 32)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint4 ld_shared_u4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v)
{
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// The two 16-bit floats of a word, in fp32.
template <bool BF16>
__device__ __forceinline__ f32x2 unpack2(uint32_t w)
{
    if constexpr (BF16) return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return pair(__half2float(__ushort_as_half(static_cast<unsigned short>(w & 0xFFFFu))),
                __half2float(__ushort_as_half(static_cast<unsigned short>(w >> 16))));
}

// A pair of fp32 values rounded to a word of two 16-bit floats.
template <bool BF16>
__device__ __forceinline__ uint32_t round2(f32x2 v)
{
    float lo, hi;
    split(v, lo, hi);
    return pack2<BF16>(__float_as_uint(lo), __float_as_uint(hi));
}

// Elements [col, col + 64) of a 16-bit row, two per word; zeros from column N on.
__device__ __forceinline__ void load_row16(uint32_t (&r)[32], const uint16_t* row, int32_t col, int32_t N)
{
    row += col;
    if (col + 64 <= N) {
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
            const uint4 v = reinterpret_cast<const uint4*>(row)[ch];
            r[4 * ch] = v.x;
            r[4 * ch + 1] = v.y;
            r[4 * ch + 2] = v.z;
            r[4 * ch + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            r[i] = col + 2 * i < N ? row[2 * i] : 0u;
            if (col + 2 * i + 1 < N) r[i] |= static_cast<uint32_t>(row[2 * i + 1]) << 16;
        }
    }
}

// Elements [col, col + 32) of an fp32 row; zeros from column N on.
__device__ __forceinline__ void load_row32(float (&r)[32], const float* row, int32_t col, int32_t N)
{
    row += col;
    if (col + 32 <= N) {
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
            const float4 v = reinterpret_cast<const float4*>(row)[ch];
            r[4 * ch] = v.x;
            r[4 * ch + 1] = v.y;
            r[4 * ch + 2] = v.z;
            r[4 * ch + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) r[i] = col + i < N ? row[i] : 0.0f;
    }
}

// Address of 16-byte chunk ch of row `lane` in a staging buffer (128-byte swizzle).
__device__ __forceinline__ uint32_t box_chunk(uint32_t stg, int lane, int ch)
{
    return stg + lane * 128 + ((ch ^ (lane & 7)) << 4);
}

// TMA store of a staging buffer that the warp has just written.
__device__ __forceinline__ void store_box_now(const CUtensorMap* tm, uint32_t stg, int32_t x, int32_t y, int lane)
{
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        ptx::tma_store_2d(tm, stg, x, y);
        ptx::bulk_commit_group();
    }
}

// Write a warp's box (lane = row y + lane, 128 bytes from column x: h) through its staging buffer
// and a TMA store, which drops rows >= M and columns >= N.  TMA clips columns to 16-byte
// granules only, so a box that straddles a ragged N is written with masked stores.
template <int ELEM>
__device__ __forceinline__ void store_rows(const uint32_t (&h)[32], int32_t x, int32_t y, int lane, uint32_t stg,
                                           const CUtensorMap* tm, void* base, int64_t ld, int32_t M, int32_t N)
{
    constexpr int kPerChunk = 16 / ELEM;   // elements of 16 bytes
    constexpr int kCols = 128 / ELEM;
    if (N % kPerChunk != 0 && x + kCols > N) {
        const int64_t row = static_cast<int64_t>(y) + lane;
        if (row < M) {
            uint8_t* dst = static_cast<uint8_t*>(base) + (row * ld + x) * ELEM;
#pragma unroll
            for (int ch = 0; ch < 8; ++ch) {
                const int32_t col = x + ch * kPerChunk;
                if (col + kPerChunk <= N) {
                    *reinterpret_cast<uint4*>(dst + ch * 16) = make_uint4(h[4 * ch], h[4 * ch + 1], h[4 * ch + 2], h[4 * ch + 3]);
                } else {
#pragma unroll
                    for (int e = 0; e < kPerChunk; ++e)
                        if (col + e < N) {
                            if constexpr (ELEM == 2)
                                reinterpret_cast<uint16_t*>(dst)[8 * ch + e] = half_of(h, 8 * ch + e);
                            else
                                reinterpret_cast<uint32_t*>(dst)[4 * ch + e] = h[4 * ch + e];
                        }
                }
            }
        }
        return;
    }
    if (lane == 0) ptx::bulk_wait_group_read<0>();  // the last store has read the buffer
    __syncwarp();
#pragma unroll
    for (int ch = 0; ch < 8; ++ch)
        ptx::st_shared_v4(box_chunk(stg, lane, ch), h[4 * ch], h[4 * ch + 1], h[4 * ch + 2], h[4 * ch + 3]);
    store_box_now(tm, stg, x, y, lane);
}

// Sums over the warp's 32 rows of 64 columns held one row per lane: lane l ends with columns 2l, 2l + 1
// in v[0], v[1].  Each step exchanges half of the columns still held with the lane `off` away.
__device__ __forceinline__ void sum_rows(float* v, int lane)
{
#pragma unroll
    for (int off = 16, n = 32; off > 0; off >>= 1, n >>= 1) {
        const bool upper = (lane & off) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = upper ? v[i] : v[i + n];
            const float keep = upper ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, off);
        }
    }
}

// tile_coord in 32 bits (a launch has fewer than 2^31 tiles): 64-bit divisions for every item took the
// epilogue warps more instructions than a relu.
__device__ __forceinline__ void tile_coord32(uint32_t t, const KernelParams& p, uint32_t& tm, uint32_t& tn)
{
    const uint32_t group_m = p.group_m, per_group = group_m * p.tiles_n;
    const uint32_t g = t / per_group, first_m = g * group_m, left = p.tiles_m - first_m;
    const uint32_t rows = left < group_m ? left : group_m;
    const uint32_t r = t - g * per_group;
    tn = r / rows;
    tm = first_m + (r - tn * rows);
}

// IN: operand type (Operand<IN>: 0 fp16, 1 bf16, 2 E4M3, 3 E5M2); OUT: kOut*; MODE: kForward, kDgrad,
// kWgrad; SUMS: the contraction runs in chunks that are summed in registers; CLUSTER: 1 (one CTA) or 2 (a CTA pair).
template <int BN, int STAGES, int IN, int OUT, int MODE, bool SUMS, int CLUSTER>
__global__ void __launch_bounds__(kTileThreads, 1)
    linear_tile_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmZ, const TileParams p)
{
    using T = Operand<IN>;
    static_assert(IN <= 3 && (BN == 128 || BN == 256), "dense operands, 64 or 128 columns per epilogue warp");
    static_assert(MODE == kForward || !T::kF8, "8-bit operands: forward only");
    static_assert(OUT != kOutF32 || (MODE == kWgrad && SUMS), "fp32 output: weight gradients only");
    constexpr bool PAIR = CLUSTER == 2;
    constexpr bool AT = MODE == kWgrad;        // A is M-major
    constexpr bool BT = MODE != kForward;      // B is N-major
    constexpr int kRanks = PAIR ? 2 : 1;
    constexpr int kTileM = kBM * kRanks;
    constexpr int kBRows = BN / kRanks;
    constexpr int CW = BN / 2;                 // columns per epilogue warp
    constexpr uint32_t kTmemCols = 2 * BN;
    using L = TileSmem<kBRows, STAGES, MODE == kDgrad ? 2 : 1>;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    uint8_t* const smem = smem_raw + (base - raw_addr);
    const uint32_t bar0 = base + L::kBarOff;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto accf_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + b); };
    auto acce_bar = [&](int b) { return bar0 + 8u * (2 * STAGES + 2 + b); };
    const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 4);
    auto in_bar = [&](int w, int b) { return bar0 + 8u * (2 * STAGES + 5 + 2 * w + b); };  // dgrad: box loaded
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
    volatile int32_t* const abort_flag = reinterpret_cast<volatile int32_t*>(smem + L::kMiscOff + 4);
    volatile int32_t* const last_flag = reinterpret_cast<volatile int32_t*>(smem + L::kMiscOff + 8);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? ptx::cluster_ctarank() : 0u;  // 0: the leader, which issues the pair's MMAs
    const bool leader = rank == 0;
    const int64_t unit = PAIR ? static_cast<int64_t>(ptx::cluster_id_x()) : static_cast<int64_t>(blockIdx.x);
    const int64_t units = PAIR ? static_cast<int64_t>(ptx::num_clusters_x()) : static_cast<int64_t>(gridDim.x);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            ptx::mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(accf_bar(b), 1);
            ptx::mbar_init(acce_bar(b), kTileEpiWarps * kRanks);
        }
        ptx::mbar_init(drain_bar, 1);
        if constexpr (MODE == kDgrad)
            for (int w = 0; w < kTileEpiWarps; ++w)
                for (int b = 0; b < 2; ++b) ptx::mbar_init(in_bar(w, b), 1);
        *abort_flag = 0;
        *last_flag = 0;
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&tmA);
        ptx::prefetch_tmap(&tmB);
        ptx::prefetch_tmap(&tmC);
    }
    __syncwarp();
    if (warp == kMmaWarp) {
        if constexpr (PAIR) {
            ptx::tmem_alloc_pair(ptx::smem_addr(tmem_slot), kTmemCols);
            ptx::tmem_relinquish_pair();
        } else {
            ptx::tmem_alloc(ptx::smem_addr(tmem_slot), kTmemCols);
            ptx::tmem_relinquish();
        }
    }
    ptx::tc_fence_before_sync();
    if constexpr (PAIR)
        ptx::cluster_sync();
    else
        __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    // Global memory waits for the stream's previous kernel.
    ptx::grid_dependency_wait();
    ptx::launch_dependents();

    Watchdog wd{abort_flag, &p};
    if constexpr (PAIR) wd.peer_abort = ptx::mapa_shared(ptx::smem_addr(const_cast<int32_t*>(abort_flag)), rank ^ 1u);

    if (warp < kTileEpiWarp0) registers_down<kTileMainRegs>();
    if (warp == kProducerWarp) {
        if (lane == 0) {
            // ---------------------------------------------------------------- producer
            uint32_t armed_mask = 0, armed_parity = 0;  // leader: stages armed, last parity
            int stage = 0;
            uint32_t phase = 0;
            int64_t loaded = 0;
            WorkIter it(p, unit, units);
            int64_t tile;
            int kb0, kb1;
            while (it.next(p, tile, kb0, kb1)) {
                uint32_t tm, tn;
                tile_coord32(static_cast<uint32_t>(tile), p, tm, tn);
                const int32_t y_a = static_cast<int32_t>(tm * kTileM + rank * kBM);
                const int32_t n_b = static_cast<int32_t>(tn * BN + rank * kBRows);
                const bool rev = it.reversed(p);
                for (int i = 0; i < kb1 - kb0; ++i, ++loaded) {
                    const int kb = rev ? kb1 - 1 - i : kb0 + i;
                    if (!wd.wait(empty_bar(stage), phase ^ 1u, kRoleProducer, tile, kb)) goto producer_done;
                    // Test hook: the first unit leaves its first stage unloaded and unarmed.
                    if (!(p.fault_inject && unit == 0 && loaded == 0)) {
                        const uint32_t sa = base + stage * L::kStageBytes;
                        const uint32_t sb = sa + L::kABytes;
                        const int32_t k0 = kb * T::kStageK;
                        const uint32_t fb = PAIR ? ptx::mapa_shared(full_bar(stage), 0u) : full_bar(stage);
                        if (leader) {
                            ptx::mbar_arrive_expect_tx(full_bar(stage), kRanks * L::kStageBytes);
                            armed_mask |= 1u << stage;
                            armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
                        }
                        auto load = [&](uint32_t dst, const CUtensorMap* tm_, int32_t x, int32_t y) {
                            if constexpr (PAIR)
                                ptx::tma_load_2d_pair(dst, tm_, x, y, fb);
                            else
                                ptx::tma_load_2d(dst, tm_, x, y, fb);
                        };
                        if constexpr (AT) {
                            // A stored contraction x rows: boxes of 64 rows (128 bytes) by kStageK contraction rows.
#pragma unroll
                            for (int q = 0; q < kBM / T::kNBlock; ++q)
                                load(sa + q * (T::kStageK * 128), &tmA, y_a + q * T::kNBlock, k0);
                        } else {
                            load(sa, &tmA, k0, y_a);
                        }
                        if constexpr (BT) {
#pragma unroll
                            for (int q = 0; q < kBRows / T::kNBlock; ++q)
                                load(sb + q * (T::kStageK * 128), &tmB, n_b + q * T::kNBlock, k0);
                        } else {
                            load(sb, &tmB, k0, n_b);
                        }
                    }
                    if (++stage == STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // Tail: every stage released, so no commit's arrival is still heading for this CTA.
            for (int i = 0; i < STAGES; ++i) {
                if (!wd.wait(empty_bar(stage), phase ^ 1u, kRoleProducer, -1, i)) goto producer_done;
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        producer_done:
            // The leader's full barriers count every load of the CTA (pair).
            if (leader)
                for (int s = 0; s < STAGES; ++s)
                    if (armed_mask & (1u << s)) wd.drain(full_bar(s), (armed_parity >> s) & 1u);
        }
    } else if (warp == kMmaWarp) {
        if (lane == 0 && leader) {
            // ---------------------------------------------------------------- MMA issuer
            constexpr uint32_t idesc = idesc_mma<T::kFormat, BT, kTileM, BN>() | (AT ? 1u << 15 : 0u);
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            bool aborted = false;
            WorkIter it(p, unit, units);
            int64_t tile;
            int kb0, kb1;
            while (!aborted && it.next(p, tile, kb0, kb1)) {
                // A loop over chunks around one over K blocks: with the chunk's wait and commit as conditions inside a
                // single loop, each K block's issue took about 60 cycles longer (8192^3 bf16: 623 against 563 us).
                const int n = kb1 - kb0;
                for (int c0 = 0; c0 < n && !aborted;) {
                    if (!wd.wait(acce_bar(acc), acc_phase ^ 1u, kRoleMma, tile, -1)) {
                        aborted = true;
                        break;
                    }
                    ptx::tc_fence_after_sync();
                    const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
                    const int c1 = n - c0 > p.chunk_kb ? c0 + p.chunk_kb : n;
                    for (int i = c0; i < c1; ++i) {
                        if (!wd.wait(full_bar(stage), phase, kRoleMma, tile, kb0 + i)) {
                            aborted = true;
                            break;
                        }
                        ptx::tc_fence_after_sync();
                        const uint32_t sa = base + stage * L::kStageBytes;
                        const uint32_t sb = sa + L::kABytes;
#pragma unroll
                        for (int k = 0; k < T::kStageK / T::kMmaK; ++k) {
                            // K-major: the k-th slice starts 32 bytes further along each 128-byte row.  M- or
                            // N-major: rows are the contraction, the k-th slice starts kMmaK rows of 128 bytes on, and
                            // 64-wide blocks are kStageK rows apart.
                            const uint64_t adesc = AT ? smem_desc_sw128(sa + k * (T::kMmaK * 128), T::kStageK * 128, 1024)
                                                      : smem_desc_sw128(sa + k * 32, 16, 1024);
                            const uint64_t bdesc = BT ? smem_desc_sw128(sb + k * (T::kMmaK * 128), T::kStageK * 128, 1024)
                                                      : smem_desc_sw128(sb + k * 32, 16, 1024);
                            const uint32_t accumulate = (i != c0 || k != 0) ? 1u : 0u;
                            if constexpr (PAIR) {
                                if constexpr (T::kF8)
                                    ptx::mma_f8_pair(d_tmem, adesc, bdesc, idesc, accumulate);
                                else
                                    ptx::mma_f16_pair(d_tmem, adesc, bdesc, idesc, accumulate);
                            } else {
                                if constexpr (T::kF8)
                                    ptx::mma_f8_cta1(d_tmem, adesc, bdesc, idesc, accumulate);
                                else
                                    ptx::mma_f16_cta1(d_tmem, adesc, bdesc, idesc, accumulate);
                            }
                        }
                        if constexpr (PAIR)
                            ptx::mma_commit_pair(empty_bar(stage), 0x3);
                        else
                            ptx::mma_commit_cta1(empty_bar(stage));
                        if (++stage == STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (aborted) break;
                    if constexpr (PAIR)
                        ptx::mma_commit_pair(accf_bar(acc), 0x3);
                    else
                        ptx::mma_commit_cta1(accf_bar(acc));
                    c0 = c1;
                    acc ^= 1;
                    if (acc == 0) acc_phase ^= 1u;
                }
            }
            if (aborted) {
                // Let every MMA issued so far finish before the TMEM is released.
                if constexpr (PAIR)
                    ptx::mma_commit_pair(drain_bar, static_cast<uint16_t>(1u << rank));
                else
                    ptx::mma_commit_cta1(drain_bar);
                wd.drain(drain_bar, 0);
            }
        }
        __syncwarp();
    } else if (warp >= kTileEpiWarp0) {
        // -------------------------------------------------------------------- epilogue
        registers_up<kTileEpiRegs>();
        const int ew = warp - kTileEpiWarp0;     // 0..7
        const int quad = warp & 3;               // TMEM lane quadrant this warp may read
        const int half = ew >> 2;                // which BN/2 columns of the tile
        const int row_in_cta = quad * 32 + lane;
        const uint32_t stg = base + L::kStgOff + ew * L::kStgBufs * kTileStgBytes;
        const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
        constexpr bool kBf16 = OUT == kOutBf16;
        int acc = 0;
        uint32_t acc_phase = 0;
        WorkIter it(p, unit, units);

        // dgrad: pre-activations come by TMA, box by box, into the staging buffer that the box's result will leave
        // from.  For whole tiles the loads run one box ahead, in the order in which finish_box takes the boxes; a tile
        // that was shared out loads its boxes when its sums are ready.  (Loaded from global memory by the lanes, 16
        // bytes of 32 rows at a time, they bound the kernel: 16384 x 1024 x 8192 relu 233 us against 176 without.)
        int in_buf = 0;                        // buffer of the next box
        uint32_t in_phase = 0, in_flight = 0;  // per buffer: parity its barrier completes next; a load is pending
        auto load_in = [&](int buf, int32_t x, int32_t y) {
            in_flight |= 1u << buf;
            if (lane == 0) {
                ptx::mbar_arrive_expect_tx(in_bar(ew, buf), kTileStgBytes);
                ptx::tma_load_2d(stg + buf * kTileStgBytes, &tmZ, x, y, in_bar(ew, buf));
            }
        };
        // A work item as this warp sees it: columns from x, rows from y of C; inside: it has some of both.
        struct Item {
            int64_t tile;
            int kb0, kb1;
            int32_t x, y;
            bool whole, inside;
        };
        auto next_item = [&](Item& t) -> bool {
            if (!it.next(p, t.tile, t.kb0, t.kb1)) return false;
            uint32_t tm, tn;
            tile_coord32(static_cast<uint32_t>(t.tile), p, tm, tn);
            t.y = static_cast<int32_t>(tm * kTileM + rank * kBM + quad * 32);
            t.x = static_cast<int32_t>(tn * BN + half * CW);
            t.whole = t.kb0 == 0 && t.kb1 == p.num_kb;
            t.inside = t.y < p.M && t.x < p.N;
            return true;
        };
        Item cur = {}, nxt = {};
        bool more_items = false;  // nxt is an item

        // The operator on 64 columns (32 for an fp32 output) of this thread's row, from column x of C on: v holds
        // the product's sums and is overwritten.  A warp's rows start at y < M, its columns at x < N.
        auto finish_box = [&](float* v, int32_t x, int32_t y) {
            const int64_t row = static_cast<int64_t>(y) + lane;
            const bool row_in = row < p.M;
            const f32x2 alpha = both(p.alpha);
            if constexpr (OUT == kOutF32) {
                uint32_t h[32];
                float r[32];
                if (p.in && row_in) {
                    load_row32(r, static_cast<const float*>(p.in) + row * p.ldin, x, p.N);
#pragma unroll
                    for (int i = 0; i < 32; ++i) h[i] = __float_as_uint(fmaf(p.beta, r[i], p.alpha * v[i]));
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) h[i] = __float_as_uint(p.alpha * v[i]);
                }
                store_rows<4>(h, x, y, lane, stg, &tmC, p.C, p.ldc, p.M, p.N);
            } else if constexpr (MODE == kDgrad) {
                // The box's pre-activations are in (or on their way to) this box's staging buffer: each 16-byte chunk
                // is read, its eight values of d rounded and written back in place, which keeps few registers alive.
                const uint32_t buf = stg + in_buf * kTileStgBytes;
                const bool has_in = p.in != nullptr;
                f32x2 w[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) w[i] = mul2(alpha, pair(v[2 * i], v[2 * i + 1]));
                if (has_in) {
                    if (!(in_flight & (1u << in_buf))) {
                        if (lane == 0) ptx::bulk_wait_group_read<0>();
                        __syncwarp();
                        load_in(in_buf, x, y);
                    }
                    const bool in = wd.wait(in_bar(ew, in_buf), (in_phase >> in_buf) & 1u, kRoleEpilogue, -1, 0);
                    if (!__all_sync(0xFFFFFFFFu, in)) return;  // recorded: the launch is being abandoned
                    in_phase ^= 1u << in_buf;
                    in_flight &= ~(1u << in_buf);
                    DTG_ACT_SWITCH(p.act, {
                        _Pragma("unroll") for (int ch = 0; ch < 8; ++ch)
                        {
                            const uint4 z = ld_shared_u4(box_chunk(buf, lane, ch));
                            w[4 * ch] = mul2(w[4 * ch], act_slope2<ACT>(unpack2<kBf16>(z.x)));
                            w[4 * ch + 1] = mul2(w[4 * ch + 1], act_slope2<ACT>(unpack2<kBf16>(z.y)));
                            w[4 * ch + 2] = mul2(w[4 * ch + 2], act_slope2<ACT>(unpack2<kBf16>(z.z)));
                            w[4 * ch + 3] = mul2(w[4 * ch + 3], act_slope2<ACT>(unpack2<kBf16>(z.w)));
                        }
                    });
                }
                // The store issued one box ago has had this box's arithmetic to read its buffer, which the next box's
                // pre-activations take: of this tile, or of the next item if that is a whole tile.  Without any, the
                // buffers alternate from TMA store to TMA store: the newest group has read the other buffer.
                const bool same_tile = x + 64 < p.N && x - cur.x + 64 < CW;
                if (has_in && (same_tile || (more_items && nxt.whole && nxt.inside))) {
                    if (lane == 0) ptx::bulk_wait_group_read<0>();
                    __syncwarp();
                    load_in(in_buf ^ 1, same_tile ? x + 64 : nxt.x, same_tile ? y : nxt.y);
                } else {
                    if (lane == 0) ptx::bulk_wait_group_read<1>();
                    __syncwarp();
                }
                const bool masked = (p.N & 7) != 0 && x + 64 > p.N;
                if (masked) {
                    uint32_t h[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) h[i] = round2<kBf16>(w[i]);
                    store_rows<2>(h, x, y, lane, buf, &tmC, p.C, p.ldc, p.M, p.N);  // its masked stores
                } else {
#pragma unroll
                    for (int ch = 0; ch < 8; ++ch)
                        ptx::st_shared_v4(box_chunk(buf, lane, ch), round2<kBf16>(w[4 * ch]), round2<kBf16>(w[4 * ch + 1]),
                                          round2<kBf16>(w[4 * ch + 2]), round2<kBf16>(w[4 * ch + 3]));
                    store_box_now(&tmC, buf, x, y, lane);
                }
                // A masked box leaves its buffer as it was and commits no group: without pre-activations the next box takes
                // the same buffer, so that waiting for all groups but the newest keeps covering it.
                if (has_in || !masked) in_buf ^= 1;
                if (p.partials) {
                    // Rows past M are not part of the sums (an infinite weight makes them NaN).
                    if (!row_in) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) w[i] = 0;
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) split(w[i], v[2 * i], v[2 * i + 1]);
                    sum_rows(v, lane);
                    *reinterpret_cast<float2*>(p.partials + static_cast<int64_t>(y >> 5) * p.pitch + x + 2 * lane) =
                        make_float2(v[0], v[1]);
                }
            } else {
                uint32_t r[32];
                const bool has_in = p.in != nullptr;
                if (has_in && row_in) {
                    load_row16(r, static_cast<const uint16_t*>(p.in) + row * p.ldin, x, p.N);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) r[i] = 0;
                }
                f32x2 w[32];
                if (MODE == kForward && p.bias) {
                    // The box's 64 biases go through the staging buffer, from which all lanes read them.
                    if (lane == 0) ptx::bulk_wait_group_read<0>();
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int32_t c = x + lane + 32 * e;
                        float f = 0.0f;
                        if (c < p.N)
                            f = p.bias_f32 ? static_cast<const float*>(p.bias)[c]
                                           : load16<kBf16>(static_cast<const uint16_t*>(p.bias) + c);
                        st_shared_f32(stg + 4 * (lane + 32 * e), f);
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float4 f = ld_shared_f4(stg + 16 * i);
                        w[2 * i] = fma2(alpha, pair(v[4 * i], v[4 * i + 1]), pair(f.x, f.y));
                        w[2 * i + 1] = fma2(alpha, pair(v[4 * i + 2], v[4 * i + 3]), pair(f.z, f.w));
                    }
                    __syncwarp();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) w[i] = mul2(alpha, pair(v[2 * i], v[2 * i + 1]));
                }
                uint32_t h[32];
                if constexpr (MODE == kForward) {
                    if (p.Z) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) h[i] = round2<kBf16>(w[i]);
                        store_rows<2>(h, x, y, lane, stg, &tmZ, p.Z, p.ldz, p.M, p.N);
                    }
                    DTG_ACT_SWITCH(p.act, {
                        _Pragma("unroll") for (int i = 0; i < 32; ++i) w[i] = act_value2<ACT>(w[i]);
                    });
                    if (has_in) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) w[i] = add2(w[i], unpack2<kBf16>(r[i]));
                    }
                }
                if constexpr (MODE == kWgrad) {
                    if (has_in) {
                        const f32x2 beta = both(p.beta);
#pragma unroll
                        for (int i = 0; i < 32; ++i) w[i] = fma2(beta, unpack2<kBf16>(r[i]), w[i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) h[i] = round2<kBf16>(w[i]);
                store_rows<2>(h, x, y, lane, stg, &tmC, p.C, p.ldc, p.M, p.N);
            }
        };

        // 64 columns of the accumulator: TMEM -> v.
        auto load_acc = [&](float* v, uint32_t taddr) {
            uint32_t a[32];
            uint32_t b[32];
            __syncwarp();
            ptx::tmem_ld_32x32b_x32(taddr, a);
            ptx::tmem_ld_32x32b_x32(taddr + 32, b);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                v[i] = __uint_as_float(a[i]);
                v[32 + i] = __uint_as_float(b[i]);
            }
        };
        auto release_acc = [&]() {
            ptx::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR)
                    ptx::mbar_arrive_cluster(ptx::mapa_shared(acce_bar(acc), 0u));
                else
                    ptx::mbar_arrive(acce_bar(acc));
            }
        };

        // Stream-K bookkeeping (see gemm_tcgen05_kernel): slots of partial sums, float4 groups of four columns with
        // the rows inner.  A part parks its sums and counts itself in; the last one to arrive adds all of them in K
        // order, whatever the order of arrival.
        constexpr size_t kSlotF4 = static_cast<size_t>(kBM) * BN / 4;
        auto slot_f4 = [&](int64_t slot) {
            return reinterpret_cast<float4*>(p.ws) + (static_cast<size_t>(slot) * CLUSTER + rank) * kSlotF4 +
                   static_cast<size_t>(half * (CW / 4)) * kBM + row_in_cta;
        };
        auto count_in = [&](int64_t tr, int64_t parts) -> bool {  // true for the part that arrives last
            __threadfence();
            tile_epi_sync();
            if (ew == 0 && lane == 0) {
                int32_t* const counter = p.counters + tr * CLUSTER + rank;
                const bool last = atomicAdd(counter, 1) == parts - 1;
                if (last) {
                    *counter = 0;  // ready for the next launch
                    __threadfence();
                }
                *last_flag = last ? 1 : 0;
            }
            tile_epi_sync();
            return *last_flag != 0;
        };
        // Has the other part of a tile of two come in already?  Then this one need not be parked: two parts give
        // the same sum in either order (v + 0 first, as a join of parked parts starts from 0: the sign of a zero).
        auto other_is_in = [&](int64_t tr, int64_t parts) -> bool {
            if (ew == 0 && lane == 0) {
                int32_t* const counter = p.counters + tr * CLUSTER + rank;
                const bool in = parts == 2 && atomicAdd(counter, 0) == 1;
                if (in) {
                    *counter = 0;
                    __threadfence();
                }
                *last_flag = in ? 1 : 0;
            }
            tile_epi_sync();
            return *last_flag != 0;
        };
        auto add_part = [&](float* v, const float4* f4) {  // 64 columns of a slot
#pragma unroll
            for (int q0 = 0; q0 < 16; q0 += 8) {
                float4 f[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) f[q] = __ldcg(f4 + (q0 + q) * kBM);
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    v[4 * (q0 + q)] += f[q].x;
                    v[4 * (q0 + q) + 1] += f[q].y;
                    v[4 * (q0 + q) + 2] += f[q].z;
                    v[4 * (q0 + q) + 3] += f[q].w;
                }
            }
        };

        // The item `cur`; false when the launch is being abandoned.
        auto one_item = [&]() -> bool {
            const int64_t tile = cur.tile;
            const int kb0 = cur.kb0, kb1 = cur.kb1;
            const int32_t y = cur.y, x0 = cur.x;
            const bool whole = cur.whole;
            const int64_t tr = tile - p.dp_tiles;
            int64_t first_unit = 0, parts = 0;
            if (!whole) sk_parts(p, tr, first_unit, parts);
            if constexpr (SUMS) {
                float s[CW];  // the running sums
                bool ok = true;
#pragma unroll
                for (int i = 0; i < CW; ++i) s[i] = 0.0f;
                for (int kb = kb0; kb < kb1; kb += p.chunk_kb) {
                    ok = ok && wd.wait(accf_bar(acc), acc_phase, kRoleEpilogue, tile, kb);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (ok) {
                        ptx::tc_fence_after_sync();
                        const uint32_t tacc = tmem_base + lane_off + static_cast<uint32_t>(acc * BN + half * CW);
#pragma unroll
                        for (int q = 0; q < CW / 32; ++q) {
                            uint32_t v[32];
                            ptx::tmem_ld_32x32b_x32(tacc + q * 32, v);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; i += 2)
                                split(add2(pair(s[q * 32 + i], s[q * 32 + i + 1]),
                                           pair(__uint_as_float(v[i]), __uint_as_float(v[i + 1]))),
                                      s[q * 32 + i], s[q * 32 + i + 1]);
                        }
                        release_acc();
                    }
                    acc ^= 1;
                    if (acc == 0) acc_phase ^= 1u;
                }
                if (!tile_epi_and(ok)) return false;
                if (!whole && other_is_in(tr, parts)) {
                    const float4* f4 = slot_f4(sk_slot(p, first_unit + (unit == first_unit ? 1 : 0), tr));
#pragma unroll
                    for (int i = 0; i < CW; ++i) s[i] += 0.0f;
#pragma unroll
                    for (int b = 0; b < CW / 64; ++b) add_part(&s[b * 64], f4 + b * 16 * kBM);
                } else if (!whole) {
                    float4* const mine = slot_f4(sk_slot(p, unit, tr));
#pragma unroll
                    for (int q = 0; q < CW / 4; ++q)
                        mine[q * kBM] = make_float4(s[4 * q], s[4 * q + 1], s[4 * q + 2], s[4 * q + 3]);
                    if (!count_in(tr, parts)) return true;
#pragma unroll
                    for (int i = 0; i < CW; ++i) s[i] = 0.0f;
                    for (int64_t part = 0; part < parts; ++part) {
                        const float4* f4 = slot_f4(sk_slot(p, first_unit + part, tr));
#pragma unroll
                        for (int b = 0; b < CW / 64; ++b) add_part(&s[b * 64], f4 + b * 16 * kBM);
                    }
                }
                if (y < p.M) {
                    constexpr int kBox = OUT == kOutF32 ? 32 : 64;
#pragma unroll
                    for (int b = 0; b < CW / kBox; ++b)
                        if (x0 + b * kBox < p.N) finish_box(&s[b * kBox], x0 + b * kBox, y);
                }
            } else {
                // One chunk: every box goes straight from the accumulator (or from the parts) to the output.
                const bool ok = kb0 == kb1 || wd.wait(accf_bar(acc), acc_phase, kRoleEpilogue, tile, kb0);
                if (!tile_epi_and(ok)) return false;
                ptx::tc_fence_after_sync();
                const uint32_t tacc = tmem_base + lane_off + static_cast<uint32_t>(acc * BN + half * CW);
                float v[64];
                if (whole) {
#pragma unroll 1
                    for (int b = 0; b < CW / 64; ++b) {
                        if (kb0 == kb1) {  // an empty contraction
#pragma unroll
                            for (int i = 0; i < 64; ++i) v[i] = 0.0f;
                        } else {
                            load_acc(v, tacc + b * 64);
                            if (b == CW / 64 - 1) release_acc();
                        }
                        if (y < p.M && x0 + b * 64 < p.N) finish_box(v, x0 + b * 64, y);
                    }
                } else if (other_is_in(tr, parts)) {
                    const float4* f4 = slot_f4(sk_slot(p, first_unit + (unit == first_unit ? 1 : 0), tr));
#pragma unroll 1
                    for (int b = 0; b < CW / 64; ++b) {
                        load_acc(v, tacc + b * 64);
                        if (b == CW / 64 - 1) release_acc();
#pragma unroll
                        for (int i = 0; i < 64; ++i) v[i] += 0.0f;
                        add_part(v, f4 + b * 16 * kBM);
                        if (y < p.M && x0 + b * 64 < p.N) finish_box(v, x0 + b * 64, y);
                    }
                } else {
                    float4* const mine = slot_f4(sk_slot(p, unit, tr));
#pragma unroll 1
                    for (int b = 0; b < CW / 64; ++b) {
                        load_acc(v, tacc + b * 64);
#pragma unroll
                        for (int q = 0; q < 16; ++q)
                            mine[(b * 16 + q) * kBM] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                    }
                    release_acc();
                    if (count_in(tr, parts)) {
#pragma unroll 1
                        for (int b = 0; b < CW / 64; ++b) {
#pragma unroll
                            for (int i = 0; i < 64; ++i) v[i] = 0.0f;
                            for (int64_t part = 0; part < parts; ++part)
                                add_part(v, slot_f4(sk_slot(p, first_unit + part, tr)) + b * 16 * kBM);
                            if (y < p.M && x0 + b * 64 < p.N) finish_box(v, x0 + b * 64, y);
                        }
                    }
                }
                if (kb0 < kb1) {
                    acc ^= 1;
                    if (acc == 0) acc_phase ^= 1u;
                }
            }
            return true;
        };

        // Bring the lines of `in` that this warp will read for `nxt` into L2, an item ahead.
        auto prefetch_in = [&]() {
            const int64_t row = static_cast<int64_t>(nxt.y) + lane;
            if (!p.in || !nxt.inside || row >= p.M) return;
            constexpr int kElem = OUT == kOutF32 ? 4 : 2;
            const uint8_t* line = static_cast<const uint8_t*>(p.in) + (row * p.ldin + nxt.x) * kElem;
#pragma unroll
            for (int b = 0; b < CW * kElem / 128; ++b)
                if (nxt.x + b * (128 / kElem) < p.N) asm volatile("prefetch.global.L2 [%0];" ::"l"(line + b * 128));
        };
        more_items = next_item(nxt);
        if (more_items) prefetch_in();
        while (more_items) {
            cur = nxt;
            more_items = next_item(nxt);
            if (more_items) prefetch_in();
            if (!one_item()) break;  // all eight epilogue warps leave together
        }
        if constexpr (MODE == kDgrad)  // after an abandoned launch: a load may still be on its way
            for (int b = 0; b < 2; ++b)
                if (in_flight & (1u << b)) wd.drain(in_bar(ew, b), (in_phase >> b) & 1u);
        if (lane == 0) ptx::bulk_wait_group_all();
        __syncwarp();
    }

    ptx::tc_fence_before_sync();
    __syncthreads();
    __syncwarp();
    if constexpr (PAIR) ptx::cluster_sync();  // neither CTA exits or frees TMEM while the peer may use it
    if (warp == kMmaWarp) {
        ptx::tc_fence_after_sync();
        if constexpr (PAIR)
            ptx::tmem_dealloc_pair(tmem_base, kTmemCols);
        else
            ptx::tmem_dealloc(tmem_base, kTmemCols);
    }
}

}  // namespace linear
}  // namespace dtg
