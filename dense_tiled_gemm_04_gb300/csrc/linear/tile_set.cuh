// The instantiations of linear_tile_kernel and how the host names them (one translation unit per
// operator and operand type, compiled in parallel).
#pragma once

#include "kernel_set.cuh"
#include "tile_kernel.cuh"

namespace dtg {
namespace linear {

template <int BN, int STAGES, int IN, int OUT, int MODE, bool SUMS, int CLUSTER>
KernelChoice tile_choice(int config)
{
    constexpr int kBRows = BN / CLUSTER;
    return {config, kBM * CLUSTER, BN, kBRows, Operand<IN>::kStageK, Operand<IN>::kNBlock, Operand<IN>::kAStageK,
            STAGES, CLUSTER, reinterpret_cast<const void*>(&linear_tile_kernel<BN, STAGES, IN, OUT, MODE, SUMS, CLUSTER>),
            TileSmem<kBRows, STAGES, MODE == kDgrad ? 2 : 1>::kAlloc, kTileThreads};
}

// config: GEMM_CONFIG_256x256 (3), _128x256 (1) or anything else (_128x128, 2).  dgrad gives a ring stage for its second
// set of staging buffers (a 5-stage ring measured as fast as a 6-stage one: 8192^3 forward 621 and 623 us).
template <int IN, int OUT, int MODE, bool SUMS>
KernelChoice tile_choice_for(int config)
{
    constexpr int kLess = MODE == kDgrad ? 1 : 0;
    if (config == 3) return tile_choice<256, 6 - kLess, IN, OUT, MODE, SUMS, 2>(3);
    if (config == 1) return tile_choice<256, 4 - kLess, IN, OUT, MODE, SUMS, 1>(1);
    return tile_choice<128, 6 - kLess, IN, OUT, MODE, SUMS, 1>(2);
}

KernelChoice forward_f16(int config);
KernelChoice forward_bf16(int config);
KernelChoice forward_e4m3(int config, bool out_bf16);
KernelChoice forward_e5m2(int config, bool out_bf16);
KernelChoice dgrad_f16(int config, bool sums);
KernelChoice dgrad_bf16(int config, bool sums);
KernelChoice wgrad_f16(int config, bool out_f32);
KernelChoice wgrad_bf16(int config, bool out_f32);
// 16-bit results of contractions that are summed in chunks for their length alone.
KernelChoice forward_long_f16(int config);
KernelChoice forward_long_bf16(int config);
KernelChoice forward_long_e4m3(int config, bool out_bf16);
KernelChoice forward_long_e5m2(int config, bool out_bf16);
KernelChoice wgrad_long_f16(int config);
KernelChoice wgrad_long_bf16(int config);

}  // namespace linear
}  // namespace dtg
