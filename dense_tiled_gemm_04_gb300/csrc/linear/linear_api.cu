// Host side of the linear-layer entry points of include/gemm.h: argument checks and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "cluster_set.cuh"
#include "elementwise.cuh"
#include "gemm.h"
#include "host/handle.cuh"
#include "tile_set.cuh"

using namespace dtg::host;
using dtg::KernelChoice;

namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 512;  // the edges of the last tiles still fit 32 bits
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
    const int64_t need = gemm_bias_grad_workspace_bytes(M, cols);
    if (!ws && need <= GEMM_OWN_SUMS_BYTES) return;  // the handle's
    if (!ws || ws_bytes < need)
        c.add(GEMM_ERR_INVALID_ARG);
    else if ((reinterpret_cast<uintptr_t>(ws) & 15u) != 0)
        c.add(GEMM_ERR_UNSUPPORTED);
}

int64_t sum_pitch(int64_t cols) { return cdiv(cols, kSumAlign) * kSumAlign; }

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

// Where a call's partial column sums go: the caller's workspace, or the handle's.
float* sums_of(gemm_handle_t h, void* workspace) { return workspace ? static_cast<float*>(workspace) : h->sums; }

dtg::linear::BiasGrad bias_grad(void* dbias, gemm_dtype_t t, float beta)
{
    return {dbias, t == GEMM_DTYPE_F32 ? dtg::linear::kOutF32 : (t == GEMM_DTYPE_BF16 ? dtg::linear::kOutBf16 : dtg::linear::kOutF16),
            beta};
}

// The bias gradient from `rows` rows of partial sums.
gemm_status_t launch_sums(const float* partials, int64_t rows, int64_t cols, const dtg::linear::BiasGrad& b, cudaStream_t s)
{
    return launch_after(&dtg::linear::column_sum_kernel, dim3(static_cast<unsigned>(cdiv(cols, 32))), dim3(32 * dtg::linear::kSumWarps), 0, s, partials,
                        rows, sum_pitch(cols), cols, b);
}

// One product: rows x cols over `depth`, as linear_tile_kernel names them.
struct Product {
    int mode;                  // dtg::linear::kForward, kDgrad, kWgrad
    gemm_dtype_t in, out;
    int64_t rows, cols, depth;
    const void *A, *B;
    int64_t lda, ldb;
    void* C;
    int64_t ldc;
    float alpha, beta;
    gemm_act_t act;
    const void* bias;
    gemm_dtype_t bias_dtype;
    const void* src;           // residual, pre-activations or dW; null: none
    int64_t ldsrc;
    void* Z;
    int64_t ldz;
    float* partials;
};

// K blocks per accumulation on one tensor-core accumulator, which truncates: a chain of K blocks loses about 1.2e-9 of
// its sum per product (see tile_kernel.cuh).  Where an fp32 result is wanted, 12 blocks of 64 keep that under 1e-6.  A
// result that is rounded to 16 bits takes up to 128 blocks as one chain, whose 1e-5 is 1/25 of fp16's half spacing where
// that is smallest; a longer contraction is cut into chains of at most that.
constexpr int64_t kChunkBlocks = 12, kLongChunkBlocks = 128;

bool fp32_result(const Product& q) { return q.out == GEMM_DTYPE_F32 || q.partials; }
int64_t k_blocks(const Product& q) { return cdiv(q.depth, is_f8(q.in) ? 128 : 64); }
int64_t chunk_limit(const Product& q) { return fp32_result(q) ? kChunkBlocks : kLongChunkBlocks; }

// Whether a product takes the tile kernel that sums chunks in registers.
bool summed(const Product& q) { return fp32_result(q) || k_blocks(q) > kLongChunkBlocks; }

KernelChoice tile_kernel(const Product& q, int config)
{
    using namespace dtg::linear;
    const bool bf16 = q.out == GEMM_DTYPE_BF16, sums = summed(q);
    if (q.mode == kDgrad) return bf16 ? dgrad_bf16(config, sums) : dgrad_f16(config, sums);
    if (q.mode == kWgrad) {
        const bool f32 = q.out == GEMM_DTYPE_F32;
        if (sums && !f32) return bf16 ? wgrad_long_bf16(config) : wgrad_long_f16(config);
        return q.in == GEMM_DTYPE_BF16 ? wgrad_bf16(config, f32) : wgrad_f16(config, f32);
    }
    switch (q.in) {
    case GEMM_DTYPE_BF16: return sums ? forward_long_bf16(config) : forward_bf16(config);
    case GEMM_DTYPE_E4M3: return sums ? forward_long_e4m3(config, bf16) : forward_e4m3(config, bf16);
    case GEMM_DTYPE_E5M2: return sums ? forward_long_e5m2(config, bf16) : forward_e5m2(config, bf16);
    default: return sums ? forward_long_f16(config) : forward_f16(config);
    }
}

// One of 14 operators and types, for the launch-state slots.
int operator_index(const Product& q)
{
    if (q.mode == dtg::linear::kForward)
        return is_f8(q.in) ? 2 + 2 * (q.in - GEMM_DTYPE_E4M3) + (q.out == GEMM_DTYPE_BF16) : q.in;
    if (q.mode == dtg::linear::kDgrad) return 6 + 2 * q.in + (q.partials != nullptr);
    return 10 + 2 * q.in + (q.out == GEMM_DTYPE_F32);
}

// One of 22 tile kernels of a configuration: forward 6 types x summed or not, dgrad 2 x 2, wgrad 2 x (16-bit, fp32, 16-bit
// summed).
int tile_slot(const Product& q, int config)
{
    const int sums = summed(q);
    const int kernel = q.mode == dtg::linear::kForward  ? 2 * operator_index(q) + sums
                       : q.mode == dtg::linear::kDgrad ? 12 + 2 * q.in + sums
                                                       : 16 + 3 * q.in + (q.out == GEMM_DTYPE_F32 ? 1 : 2 * sums);
    return kLinearSlot0 + 3 * kernel + (config - 1);
}

int cluster_slot(const Product& q, int tokens)
{
    return kLinearSlot0 + kLinearTileSlots + 4 * operator_index(q) + (tokens == 16 ? 0 : tokens == 32 ? 1 : tokens == 64 ? 2 : 3);
}

// Whether a product runs on linear_cluster_kernel, and how.
struct ClusterPlan {
    int tokens = 0;  // per tile; 0: the tile kernels
    int ranks = 1;   // CTAs per cluster
    int32_t chunk_kb = 0;  // K blocks per accumulator
    KernelChoice kc;
};

KernelChoice cluster_kernel(const Product& q, int tokens)
{
    using namespace dtg::linear;
    const bool bf16 = q.out == GEMM_DTYPE_BF16;
    if (q.mode == kDgrad) return cluster_dgrad(tokens, bf16);
    if (q.mode == kWgrad) return cluster_wgrad(q.in == GEMM_DTYPE_BF16, q.out == GEMM_DTYPE_F32);
    return is_f8(q.in) ? cluster_forward_8(tokens, q.in == GEMM_DTYPE_E5M2, bf16) : cluster_forward_16(tokens, bf16);
}

// Clusters of 2^log CTAs of a kernel that the GPU runs at once.  Its GPCs differ in size, so that is fewer than the
// SMs alone would say: clusters of 16 for 16 tiles took a second round, 21.3 us for 256 x 1024 x 8192 against 13.6
// with 8.  The runtime counts one CTA of these kernels per SM (76, 36, 15, 7 clusters of 2, 4, 8, 16); two run, as
// their shared memory allows: 128 x 8192 x 8192 on 64 clusters of 4 takes 28.7 us, on 64 of 2 36.2.
gemm_status_t clusters_that_fit(DeviceState& dev, const KernelChoice& kc, int slot, int log, int* n)
{
    std::lock_guard<std::mutex> lock(dev.mu);
    if (dev.fits[slot][log] == 0) {
        cudaLaunchConfig_t cfg;
        std::memset(&cfg, 0, sizeof(cfg));
        cfg.gridDim = dim3(1u << log, 1, 1);
        cfg.blockDim = dim3(static_cast<unsigned>(kc.threads), 1, 1);
        cfg.dynamicSmemBytes = static_cast<size_t>(kc.smem);
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 1u << log;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&dev.fits[slot][log], kc.fn, &cfg) != cudaSuccess) return GEMM_ERR_CUDA;
        if (dev.fits[slot][log] == 0) dev.fits[slot][log] = -1;
    }
    *n = 2 * dev.fits[slot][log];
    return GEMM_OK;
}

gemm_status_t plan_cluster(const LaunchOptions& o, DeviceState& dev, const Product& q, ClusterPlan* c)
{
    if (o.config != GEMM_CONFIG_AUTO || q.depth == 0) return GEMM_OK;
    const int64_t kb = k_blocks(q);
    int tokens = q.rows <= 16 ? 16 : q.rows <= 32 ? 32 : q.rows <= 64 ? 64 : 128;
    if (q.mode == dtg::linear::kDgrad && tokens < 64) tokens = 64;
    if (q.mode == dtg::linear::kWgrad) tokens = 128;
    // Where the tile kernels would leave SMs idle: on fewer than 128 tokens, whose narrower tiles are the cheaper ones
    // (8 x 8192 x 1024: 7.1 us, 10.6 on 128 x 128 tiles); and, in tiles of 128 tokens as large as theirs, where a
    // split gains.  On a quarter of a tile per SM or less it always does, and 64 tokens a tile do it better (256 x
    // 1024 x 1024: 5.8 us, 9.5 whole; 128 x 4096 x 4096: 12.1, 14.1 in 128).  Up to a tile per SM it does with more
    // than 16 K blocks (256 x 8192 x 8192: 37.8 us, 40.8 whole; but 2048 x 1024 x 1024: 12.3, 10.0 whole).  More
    // tiles are not split (512 x 8192 x 8192: 65 us, 47 on CTA pairs).
    int64_t tiles = cdiv(q.cols, dtg::kBM) * cdiv(q.rows, tokens);
    const int64_t slots = 2 * dev.num_sms;
    if (tokens == 128) {
        const bool few = 4 * tiles <= dev.num_sms;
        if (!few && (tiles > dev.num_sms || kb <= 16)) return GEMM_OK;
        if (few && q.mode != dtg::linear::kWgrad) {
            tokens = 64;
            tiles = cdiv(q.cols, dtg::kBM) * cdiv(q.rows, tokens);
        }
    }
    if (tiles > slots) return GEMM_OK;
    c->kc = cluster_kernel(q, tokens);
    const int slot = cluster_slot(q, tokens);
    // Clusters of 16 are beyond the portable size.
    if (!dev.attrs_set[slot] && cudaFuncSetAttribute(c->kc.fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return GEMM_ERR_CUDA;
    gemm_status_t st = ensure_kernel_ready(dev, c->kc, slot);
    // Double the ranks while every cluster still runs at once and each rank keeps two K blocks.
    int log = 0;
    while (st == GEMM_OK && (1 << log) < dtg::linear::kClusterMaxSplit && tiles * (2 << log) <= slots && kb >= (4 << log)) {
        int n = 0;
        st = clusters_that_fit(dev, c->kc, slot, log + 1, &n);
        if (n < tiles) break;
        ++log;
    }
    if (st != GEMM_OK) return st;
    // Chains of products no longer than the tile kernels', on as many accumulators as there are.
    const int64_t blocks = cdiv(kb, 1 << log), chunks = cdiv(blocks, chunk_limit(q));
    if (chunks > 256 / tokens) return GEMM_OK;
    c->chunk_kb = static_cast<int32_t>(cdiv(blocks, chunks));
    c->tokens = tokens;
    c->ranks = 1 << log;
    return GEMM_OK;
}

gemm_status_t launch_cluster(gemm_handle_t h, const Product& q, const ClusterPlan& plan, int64_t* sum_rows, cudaStream_t stream)
{
    using namespace dtg::linear;
    const KernelChoice& kc = plan.kc;
    const uint64_t eb = static_cast<uint64_t>(elem_bytes(q.in));
    const uint32_t sk = static_cast<uint32_t>(kc.stage_k), nb = static_cast<uint32_t>(kc.n_block);
    // The features' operand is B (its rows are the output's columns), the tokens' is A.
    CUtensorMap tF, tT;
    if (!(q.mode == kForward ? get_tmap(nullptr, q.B, q.depth, q.cols, q.ldb * eb, sk, dtg::kBM, q.in, &tF)
                             : get_tmap(nullptr, q.B, q.cols, q.depth, q.ldb * eb, nb, sk, q.in, &tF)) ||
        !(q.mode == kWgrad ? get_tmap(nullptr, q.A, q.rows, q.depth, q.lda * eb, nb, sk, q.in, &tT)
                           : get_tmap(nullptr, q.A, q.depth, q.rows, q.lda * eb, sk, static_cast<uint32_t>(plan.tokens), q.in, &tT)))
        return GEMM_ERR_CUDA;
    const int64_t tiles_t = cdiv(q.rows, plan.tokens), tiles_f = cdiv(q.cols, dtg::kBM);
    const int64_t grid = tiles_t * tiles_f * plan.ranks;
    if (sum_rows) *sum_rows = tiles_t;
    ClusterParams p;
    std::memset(&p, 0, sizeof(p));
    p.M = static_cast<int32_t>(q.rows);
    p.N = static_cast<int32_t>(q.cols);
    p.K = static_cast<int32_t>(q.depth);
    p.num_kb = static_cast<int32_t>(cdiv(q.depth, kc.stage_k));
    p.fault_inject = static_cast<int32_t>(h->opts.fault_inject);
    p.timeout_ns = static_cast<uint64_t>(h->opts.timeout_ns);
    p.err = h->d_err;
    p.C = q.C;
    p.ldc = q.ldc;
    p.alpha = q.alpha;
    p.beta = q.beta;
    p.tiles_t = static_cast<int32_t>(tiles_t);
    p.chunk_kb = plan.chunk_kb;
    p.act = q.act;
    p.bias = q.bias;
    p.bias_f32 = q.bias_dtype == GEMM_DTYPE_F32;
    p.in = q.src;
    p.ldin = q.ldsrc;
    p.Z = q.Z;
    p.ldz = q.ldz;
    p.partials = q.partials;
    p.pitch = sum_pitch(q.cols);
    void* args[] = {&tF, &tT, &p};
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(kc.threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(kc.smem);
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = static_cast<unsigned>(plan.ranks);
    attrs[1].val.clusterDim.y = 1;
    attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = 2;
    return cudaLaunchKernelExC(&cfg, kc.fn, args) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

// Enqueue a product.  sum_rows: receives the rows of partial column sums that it writes.
gemm_status_t launch_product(gemm_handle_t h, const Product& q, int64_t* sum_rows, cudaStream_t stream)
{
    const LaunchOptions& o = h->opts;
    ClusterPlan few;
    const gemm_status_t planned = plan_cluster(o, h->dev, q, &few);
    if (planned != GEMM_OK) return planned;
    if (few.tokens) return launch_cluster(h, q, few, sum_rows, stream);
    if (sum_rows) *sum_rows = cdiv(q.rows, kSumRows);
    int config = pick_config(o, h->dev, q.rows, q.cols, q.depth);
    if (config == GEMM_CONFIG_128x64) config = GEMM_CONFIG_128x128;
    // CTA pairs from 2/5 of a tile per SM on, where gemm_run asks for 1/2: on 64 pair tiles 512 x 8192 x 8192 takes 46.8
    // us against 57.7 in 128 x 256 tiles, 1024 x 4096 x 4096 27.0 and 30.7; on 32 256 x 8192 x 8192 46.2 and 40.8.
    if (o.config == GEMM_CONFIG_AUTO && cdiv(q.rows, 256) * cdiv(q.cols, 256) * 5 >= 2 * h->dev.num_sms)
        config = GEMM_CONFIG_256x256;
    const KernelChoice kc = tile_kernel(q, config);
    const int slot = tile_slot(q, kc.config);
    if (!h->dev.attrs_set[slot]) {
        // The kernel's warps share out the registers it starts with: fewer than it counts on would leave the
        // epilogue waiting for registers forever.
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, kc.fn) != cudaSuccess || fa.numRegs < dtg::linear::kTileLaunchRegs)
            return GEMM_ERR_CUDA;
    }
    const gemm_status_t ready = ensure_kernel_ready(h->dev, kc, slot);
    if (ready != GEMM_OK) return ready;
    gemm_plan_t plan;
    fill_plan(o, h->dev, h->dev.max_clusters[slot], &h->ws, q.rows, q.cols, q.depth, kc, kDense, &plan);
    // Sharing out the K blocks of the last tiles (stream-K) pays when the units that a last wave of whole tiles would
    // leave idle are worth more K blocks than the joins cost, about 56 blocks of a 256-wide 16-bit tile (16384 x 1024
    // x 8192 forward, 81 blocks a tile: 166 us shared, 174 whole; dgrad of the same, 1 block: 311 and 294).  Between
    // one and two waves the planner would share every tile, with each unit starting at another K, and the operands'
    // reuse in L2 is lost (wgrad 1024 x 8192 over 16384 tokens, 1.7 waves: 209 us shared, 190 whole; a wave of whole
    // tiles and the rest shared, under the power limit: 191).  Under one wave the planner's rule stands.
    const int64_t tiles = plan.tiles_m * plan.tiles_n, units = plan.grid / kc.cluster;
    if (plan.dp_tiles < tiles && tiles >= units) {
        const int64_t idle = cdiv(tiles, units) * units - tiles;
        const int64_t join = 56 * (256 / kc.bn) * (is_f8(q.in) ? 2 : 1);
        if (plan.dp_tiles == 0 || idle * plan.k_blocks < join * units) {
            LaunchOptions whole = o;
            whole.stream_k = 0;
            fill_plan(whole, h->dev, h->dev.max_clusters[slot], &h->ws, q.rows, q.cols, q.depth, kc, kDense, &plan);
        }
    }
    // The kernel numbers tiles, and a raster group's, in 32 bits.
    if (tiles > kMaxDim) return GEMM_ERR_UNSUPPORTED;
    plan.raster_group = std::min(plan.raster_group, plan.tiles_m);

    const uint64_t eb = static_cast<uint64_t>(elem_bytes(q.in));
    const uint32_t sk = static_cast<uint32_t>(kc.stage_k), nb = static_cast<uint32_t>(kc.n_block);
    const uint64_t oe = static_cast<uint64_t>(bytes_of(q.out));
    CUtensorMap tA, tB, tC, tZ;
    if (!get_tmap(nullptr, q.C, q.cols, q.rows, q.ldc * oe, static_cast<uint32_t>(128 / oe), 32, q.out, &tC))
        return GEMM_ERR_CUDA;
    tA = tB = tZ = tC;  // those that are not used name a valid tensor
    if (q.Z && !get_tmap(nullptr, q.Z, q.cols, q.rows, q.ldz * oe, static_cast<uint32_t>(128 / oe), 32, q.out, &tZ))
        return GEMM_ERR_CUDA;
    if (q.mode == dtg::linear::kDgrad && q.src &&  // the boxes of pre-activations: those of the output
        !get_tmap(nullptr, q.src, q.cols, q.rows, q.ldsrc * oe, static_cast<uint32_t>(128 / oe), 32, q.out, &tZ))
        return GEMM_ERR_CUDA;
    if (q.depth > 0) {
        const bool at = q.mode == dtg::linear::kWgrad, bt = q.mode != dtg::linear::kForward;
        if (!(at ? get_tmap(nullptr, q.A, q.rows, q.depth, q.lda * eb, nb, sk, q.in, &tA)
                 : get_tmap(nullptr, q.A, q.depth, q.rows, q.lda * eb, sk, dtg::kBM, q.in, &tA)) ||
            !(bt ? get_tmap(nullptr, q.B, q.cols, q.depth, q.ldb * eb, nb, sk, q.in, &tB)
                 : get_tmap(nullptr, q.B, q.depth, q.cols, q.ldb * eb, sk, static_cast<uint32_t>(kc.b_box), q.in, &tB)))
            return GEMM_ERR_CUDA;
    }

    dtg::linear::TileParams p;
    std::memset(&p, 0, sizeof(p));
    p.M = static_cast<int32_t>(q.rows);
    p.N = static_cast<int32_t>(q.cols);
    p.K = static_cast<int32_t>(q.depth);
    p.tiles_m = static_cast<int32_t>(plan.tiles_m);
    p.tiles_n = static_cast<int32_t>(plan.tiles_n);
    p.num_kb = static_cast<int32_t>(plan.k_blocks);
    p.num_tiles = static_cast<int32_t>(plan.tiles_m * plan.tiles_n);
    p.group_m = static_cast<int32_t>(plan.raster_group);
    p.fault_inject = static_cast<int32_t>(o.fault_inject);
    p.k_snake = static_cast<int32_t>(plan.k_snake);
    p.timeout_ns = static_cast<uint64_t>(o.timeout_ns);
    p.err = h->d_err;
    p.C = q.C;
    p.ldc = q.ldc;
    p.dp_tiles = static_cast<int32_t>(plan.dp_tiles);
    p.sk_base = plan.sk_base;
    p.sk_extra = plan.sk_extra;
    p.ws = h->ws.partials;
    p.counters = h->ws.counters;
    p.alpha = q.alpha;
    p.beta = q.beta;
    // SUMS kernels: chunks of equal length (within one); the others take a contraction as one chunk.
    p.chunk_kb = INT32_MAX;
    if (summed(q) && plan.k_blocks > 0)
        p.chunk_kb = static_cast<int32_t>(cdiv(plan.k_blocks, cdiv(plan.k_blocks, chunk_limit(q))));
    p.act = q.act;
    p.bias = q.bias;
    p.bias_f32 = q.bias_dtype == GEMM_DTYPE_F32;
    p.in = q.src;
    p.ldin = q.ldsrc;
    p.Z = q.Z;
    p.ldz = q.ldz;
    p.partials = q.partials;
    p.pitch = sum_pitch(q.cols);

    void* args[] = {&tA, &tB, &tC, &tZ, &p};
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>(plan.grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(kc.threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(kc.smem);
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    if (kc.cluster > 1) {
        attrs[1].id = cudaLaunchAttributeClusterDimension;
        attrs[1].val.clusterDim.x = static_cast<unsigned>(kc.cluster);
        attrs[1].val.clusterDim.y = 1;
        attrs[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    cfg.attrs = attrs;
    return cudaLaunchKernelExC(&cfg, kc.fn, args) == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA;
}

template <bool BF16>
gemm_status_t launch_act_grad(const dtg::linear::ActGradParams& p, gemm_act_t act, dim3 grid, cudaStream_t s)
{
    using namespace dtg::linear;
    void (*fn)(const ActGradParams) = nullptr;
    DTG_ACT_SWITCH(act, fn = (&act_grad_kernel<BF16, ACT>));
    return launch_after(fn, grid, dim3(kActWarps * 32), 0, s, p);
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
    Product q = {};
    q.mode = dtg::linear::kForward;
    q.in = a.dtype;
    q.out = a.out_dtype;
    q.rows = a.M;
    q.cols = a.N;
    q.depth = a.K;
    q.A = a.X;
    q.lda = a.ldx;
    q.B = a.W;
    q.ldb = a.ldw;
    q.C = a.Y;
    q.ldc = a.ldy;
    q.alpha = a.alpha;
    q.act = a.act;
    q.bias = a.bias;
    q.bias_dtype = a.bias_dtype;
    q.src = a.residual;
    q.ldsrc = a.ldr;
    q.Z = a.Z;
    q.ldz = a.ldz;
    return launch_product(h, q, nullptr, static_cast<cudaStream_t>(stream));
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
    int64_t rows = 0;  // of partial sums
    if (a.M > 0) {
        Product q = {};
        q.mode = dtg::linear::kDgrad;
        q.in = q.out = a.dtype;
        q.rows = a.M;
        q.cols = a.K;
        q.depth = a.N;
        q.A = a.dY;
        q.lda = a.lddy;
        q.B = a.W;
        q.ldb = a.ldw;
        q.C = a.dX;
        q.ldc = a.lddx;
        q.alpha = a.alpha;
        q.act = a.act;
        q.src = a.act != GEMM_ACT_NONE ? a.Z : nullptr;
        q.ldsrc = a.ldz;
        q.partials = a.dbias ? sums_of(h, a.workspace) : nullptr;
        const gemm_status_t st = launch_product(h, q, &rows, s);
        if (st != GEMM_OK) return st;
    }
    if (!a.dbias) return GEMM_OK;
    return launch_sums(sums_of(h, a.workspace), rows, a.K, bias_grad(a.dbias, a.dbias_dtype, a.beta_bias), s);
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
    Product q = {};
    q.mode = dtg::linear::kWgrad;
    q.in = a.dtype;
    q.out = a.out_dtype;
    q.rows = a.N;
    q.cols = a.K;
    q.depth = a.M;
    q.A = a.dY;
    q.lda = a.lddy;
    q.B = a.X;
    q.ldb = a.ldx;
    q.C = a.dW;
    q.ldc = a.lddw;
    q.alpha = a.alpha;
    q.beta = a.beta;
    q.src = a.beta != 0.0f ? a.dW : nullptr;
    q.ldsrc = a.lddw;
    return launch_product(h, q, nullptr, static_cast<cudaStream_t>(stream));
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
    const dtg::linear::BiasGrad bias = bias_grad(a.dbias, a.dbias_dtype, a.beta_bias);
    if (a.M == 0) return a.dbias ? launch_sums(nullptr, 0, a.N, bias, s) : GEMM_OK;
    if (!a.dZ && !a.dbias) return GEMM_OK;
    // Blocks of rows: 64, or 32 (what the workspace has room for) when those would not fill the GPU.  Up to 128
    // rows are one block, which writes dbias itself and saves the second launch.
    const int64_t strips = cdiv(a.N, dtg::linear::kActCols);
    const int64_t block_rows = a.M <= 128 ? a.M : (strips * cdiv(a.M, 64) >= 6 * h->dev.num_sms ? 64 : kSumRows);
    const int64_t blocks = cdiv(a.M, block_rows);
    const bool one_block = blocks == 1;
    dtg::linear::ActGradParams p;
    p.dY = static_cast<const uint16_t*>(a.dY);
    p.Z = static_cast<const uint16_t*>(a.Z);
    p.dZ = static_cast<uint16_t*>(a.dZ);
    p.partials = a.dbias && !one_block ? sums_of(h, a.workspace) : nullptr;
    p.bias = bias;
    p.M = a.M;
    p.N = a.N;
    p.lddy = a.lddy;
    p.ldz = a.ldz;
    p.lddz = a.lddz;
    p.pitch = sum_pitch(a.N);
    p.block_rows = block_rows;
    const dim3 grid(static_cast<unsigned>(strips), static_cast<unsigned>(std::min<int64_t>(blocks, 65535)));
    const gemm_status_t st = a.dtype == GEMM_DTYPE_BF16 ? launch_act_grad<true>(p, a.act, grid, s)
                                                        : launch_act_grad<false>(p, a.act, grid, s);
    if (st != GEMM_OK || !a.dbias || one_block) return st;
    return launch_sums(p.partials, blocks, a.N, bias, s);
}

}  // extern "C"
