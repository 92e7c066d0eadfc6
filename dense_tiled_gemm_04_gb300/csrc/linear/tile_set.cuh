// The instantiations of linear_tile_kernel and how the host names them (one translation unit per
// operator and operand type, compiled in parallel).
#pragma once

#include "kernel_set.cuh"
#include "tile_kernel.cuh"

namespace dtg {
namespace linear {

template <int BN, int STAGES, int IN, int OUT, int MODE, bool SUMS, int CLUSTER, bool SCALED = false,
          int STG_BUFS = MODE == kDgrad ? 2 : 1>
KernelChoice tile_choice(int config)
{
    constexpr int kBRows = BN / CLUSTER;
    return {config, kBM * CLUSTER, BN, kBRows, Operand<IN>::kStageK, Operand<IN>::kNBlock, Operand<IN>::kAStageK,
            STAGES, CLUSTER,
            reinterpret_cast<const void*>(&linear_tile_kernel<BN, STAGES, IN, OUT, MODE, SUMS, CLUSTER, SCALED, STG_BUFS>),
            TileSmem<kBRows, STAGES, STG_BUFS>::kAlloc, kTileThreads};
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

// 8-bit operands with block scales: a pair with 256 accumulator columns (gated: 128 of each half) or (any other config) one CTA
// with 128.
template <int OUT, int MODE>
KernelChoice scaled_choice(int config)
{
    if (config == 3) return tile_choice<256, 6, 2, OUT, MODE, true, 2, true>(3);
    return tile_choice<128, 6, 2, OUT, MODE, true, 1, true>(2);
}

// Gated forward, 16-bit operands: a pair or one CTA with 256 accumulator columns, 128 of each half.
template <int IN, int OUT, bool SUMS>
KernelChoice glu_choice(int config)
{
    if (config == 3) return tile_choice<256, 6, IN, OUT, kGlu, SUMS, 2>(3);
    return tile_choice<256, 4, IN, OUT, kGlu, SUMS, 1>(1);
}

// Gated dgrad: a ring stage given for g's and u's staging buffers.
template <int IN, int OUT, bool SUMS>
KernelChoice glu_dgrad_choice(int config)
{
    if (config == 3) return tile_choice<256, 5, IN, OUT, kGluDgrad, SUMS, 2, false, 2>(3);
    return tile_choice<256, 3, IN, OUT, kGluDgrad, SUMS, 1, false, 2>(1);
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
// Block scales (E4M3 and E5M2), and gated layers.
KernelChoice forward_scaled(int config, bool out_bf16);
KernelChoice glu_16(int config, bool bf16, bool sums);
KernelChoice glu_scaled(int config, bool out_bf16);
KernelChoice glu_dgrad_f16(int config, bool sums);
KernelChoice glu_dgrad_bf16(int config, bool sums);

}  // namespace linear
}  // namespace dtg
