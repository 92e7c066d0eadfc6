// The instantiations of linear_cluster_kernel and how the host names them.
#pragma once

#include "cluster_kernel.cuh"
#include "kernel_set.cuh"

namespace dtg {
namespace linear {

// bm: tokens per tile, bn: features; the cluster's size is chosen at launch.
template <int BN, int IN, int OUT, int MODE, bool SCALED = false>
KernelChoice cluster_choice()
{
    using L = ClusterSmem<BN, SCALED, MODE == kGluDgrad ? 2 : 1>;
    return {0, BN, MODE == kGlu ? kBM / 2 : kBM, BN, Operand<IN>::kStageK, Operand<IN>::kNBlock, Operand<IN>::kAStageK, L::kStages,
            1, reinterpret_cast<const void*>(&linear_cluster_kernel<BN, IN, OUT, MODE, SCALED>), L::kAlloc, kClusterThreads};
}

// Gated forward and block-scaled products: 16, 32 or 64 tokens.
template <int IN, int OUT, int MODE, bool SCALED>
KernelChoice cluster_choice_narrow(int tokens)
{
    if (tokens == 16) return cluster_choice<16, IN, OUT, MODE, SCALED>();
    if (tokens == 32) return cluster_choice<32, IN, OUT, MODE, SCALED>();
    return cluster_choice<64, IN, OUT, MODE, SCALED>();
}

// tokens: 16, 32, 64 or 128 per tile (wgrad: 128; dgrad: 64 or 128).
template <int IN, int OUT, int MODE>
KernelChoice cluster_choice_for(int tokens)
{
    if constexpr (MODE == kForward) {
        if (tokens == 16) return cluster_choice<16, IN, OUT, MODE>();
        if (tokens == 32) return cluster_choice<32, IN, OUT, MODE>();
    }
    if constexpr (MODE != kWgrad) {
        if (tokens == 64) return cluster_choice<64, IN, OUT, MODE>();
    }
    return cluster_choice<128, IN, OUT, MODE>();
}

KernelChoice cluster_forward_16(int tokens, bool bf16);
KernelChoice cluster_forward_8(int tokens, bool e5m2, bool out_bf16);
KernelChoice cluster_dgrad(int tokens, bool bf16);
KernelChoice cluster_wgrad(bool bf16, bool out_f32);
// tokens: 16, 32 or 64; gated dgrad: 64.
KernelChoice cluster_scaled(int tokens, bool out_bf16);
KernelChoice cluster_glu_16(int tokens, bool bf16);
KernelChoice cluster_glu_scaled(int tokens, bool out_bf16);
KernelChoice cluster_glu_dgrad(bool bf16);

}  // namespace linear
}  // namespace dtg
