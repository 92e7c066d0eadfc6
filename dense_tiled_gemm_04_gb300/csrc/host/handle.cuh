// Host-side state shared by the library's entry points: the handle, its options and workspaces, and
// the helpers (defined in gemm_api.cu) that encode tensor maps, ready kernels and plan launches.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <vector>

#include "gemm.h"
#include "kernel_set.cuh"

namespace dtg {
namespace host {

constexpr int64_t kTimeoutDefaultNs = 2000000000LL;  // 2 s per wait
// Kernels whose launch state is kept: gemm_run and its relatives (4 configurations x 12 operand /
// output types x 2 layouts), then those of the linear-layer entry points.
constexpr int kLinearSlot0 = 96;
constexpr int kLinearTileSlots = 3 * 22;     // tile kernels: operators, types and sums x tiles
constexpr int kLinearClusterSlots = 4 * 14;  // cluster kernels: operators and types x token sizes
constexpr int kNumSlots = kLinearSlot0 + kLinearTileSlots + kLinearClusterSlots;
constexpr int64_t kMinStreamKBlocks = 8;   // default shortest stream-K share (GEMM_OPT_SK_MIN_BLOCKS)
constexpr int64_t kMinSplitBlocks = 32;    // default shortest share of a split under one wave (GEMM_OPT_SPLIT_MIN_BLOCKS)

struct TmapKey {
    const void* ptr;
    uint64_t inner, outer, pitch_bytes;
    uint32_t box_inner, box_outer;
    int32_t dtype;
    int32_t swizzle;
    bool operator==(const TmapKey& o) const
    {
        return ptr == o.ptr && inner == o.inner && outer == o.outer && pitch_bytes == o.pitch_bytes &&
               box_inner == o.box_inner && box_outer == o.box_outer && dtype == o.dtype && swizzle == o.swizzle;
    }
};

struct TmapEntry {
    TmapKey key;
    CUtensorMap map;
};

// Tunables a launch reads (a handle's options, or the defaults).
struct LaunchOptions {
    int64_t config = GEMM_CONFIG_AUTO;
    int64_t timeout_ns = kTimeoutDefaultNs;
    int64_t max_ctas = 0;
    int64_t raster_group = 0;  // 0: automatic
    int64_t fault_inject = 0;
    int64_t stream_k = 1;
    int64_t sk_min_blocks = kMinStreamKBlocks;
    int64_t split_min_blocks = kMinSplitBlocks;
    int64_t k_snake = 1;
    int64_t host_row_chunks = 8;
    int64_t host_col_chunks = 4;
};

// Per-device facts and lazily-set per-kernel state.  Guarded by `mu`.
struct DeviceState {
    int num_sms = 0;
    std::mutex mu;
    bool attrs_set[kNumSlots] = {};
    int max_clusters[kNumSlots] = {};  // pair kernels: co-resident clusters (0 = not yet queried)
    int fits[kNumSlots][5] = {};       // kernels of any cluster size: those of 1, 2, 4, 8, 16 CTAs, likewise
};

// Streams and events of gemm_run_host's copy/compute pipeline (created on first use).
struct HostPipe {
    static constexpr int kMaxRowChunks = 16;  // row chunks of A (and C)
    static constexpr int kMaxColChunks = 8;   // column chunks of C (B's rows for TN, columns for NN)
    static constexpr int kMaxPieces = kMaxRowChunks + kMaxColChunks;
    bool ready = false;
    cudaStream_t in = nullptr, out = nullptr;  // host -> device copies, in order; device -> host copies
    cudaEvent_t start = nullptr, done = nullptr;
    cudaEvent_t arrived[kMaxPieces] = {};      // per input piece, in transfer order
    cudaEvent_t computed[kMaxPieces] = {};     // per GEMM launch
};

// Stream-K workspace: fp32 partial sums and arrival counters (see gemm_kernel.cuh).
struct Workspace {
    float* partials = nullptr;
    int32_t* counters = nullptr;
    size_t partial_floats = 0;  // capacity
    int64_t counter_count = 0;  // capacity
};

// Keeps the caller's current device unchanged across a call made on h->device.
struct DeviceGuard {
    int prev = -1;
    bool ok = false;
    explicit DeviceGuard(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess) return;
        ok = (prev == dev) || (cudaSetDevice(dev) == cudaSuccess);
    }
    ~DeviceGuard()
    {
        int cur = -1;
        if (prev >= 0 && cudaGetDevice(&cur) == cudaSuccess && cur != prev) cudaSetDevice(prev);
    }
};

// Encode a 2-D row-major tensor map: `inner` contiguous elements per row, `outer` rows
// `pitch_bytes` apart, box = box_inner x box_outer, 128-byte swizzle (or none), zero fill
// outside.  With a cache (a handle's), identical requests reuse the earlier encoding.
bool get_tmap(std::vector<TmapEntry>* cache, const void* ptr, uint64_t inner, uint64_t outer, uint64_t pitch_bytes,
              uint32_t box_inner, uint32_t box_outer, int32_t dtype, CUtensorMap* out,
              CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool is_f8(gemm_dtype_t t) { return t == GEMM_DTYPE_E4M3 || t == GEMM_DTYPE_E5M2; }
inline int elem_bytes(gemm_dtype_t t) { return is_f8(t) ? 1 : 2; }

// Kernel families beyond the dense one: block-scaled 8-bit operands, 2:4-sparse A (each with
// the one-CTA 128 x 256 tile and the CTA pair).
enum Family { kDense = 0, kBlockScaled = 1, kSparse24 = 2 };

// Opt the kernel into its shared memory and, for pair kernels, ask how many clusters can
// be resident at once (the persistent grid never exceeds that).  Once per device and slot.
gemm_status_t ensure_kernel_ready(DeviceState& dev, const KernelChoice& kc, int slot);

// The tile configuration for an M x N product over K (options first, then sizes).
int pick_config(const LaunchOptions& o, const DeviceState& dev, int64_t M, int64_t N, int64_t K);

// The launch of a product: grid, raster group, whole tiles and stream-K shares.
// `ws` == nullptr: no workspace, every tile is done whole (data-parallel).
void fill_plan(const LaunchOptions& o, const DeviceState& dev, int max_clusters, const Workspace* ws, int64_t M,
               int64_t N, int64_t K, const KernelChoice& kc, int family, gemm_plan_t* plan);

}  // namespace host
}  // namespace dtg

struct gemm_handle_s {
    int device = 0;
    int32_t* d_err = nullptr;  // 4 ints
    int32_t last_info[4] = {0, 0, 0, 0};
    dtg::host::LaunchOptions opts;
    dtg::host::DeviceState dev;
    dtg::host::Workspace ws;
    float* sums = nullptr;  // GEMM_OWN_SUMS_BYTES for column sums
    std::vector<dtg::host::TmapEntry> tmaps;
    // gemm_run_host staging and pipeline
    void* d_stage = nullptr;
    size_t stage_bytes = 0;
    dtg::host::HostPipe pipe;
};
