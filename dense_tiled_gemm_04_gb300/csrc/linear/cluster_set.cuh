// The instantiations of linear_cluster_kernel and how the host names them.
#pragma once

#include "cluster_kernel.cuh"
#include "kernel_set.cuh"

namespace dtg {
namespace linear {

// bm: tokens per tile, bn: features; the cluster's size is chosen at launch.
template <int BN, int IN, int OUT, int MODE>
KernelChoice cluster_choice()
{
    return {0, BN, kBM, BN, Operand<IN>::kStageK, Operand<IN>::kNBlock, Operand<IN>::kAStageK, ClusterSmem<BN>::kStages, 1,
            reinterpret_cast<const void*>(&linear_cluster_kernel<BN, IN, OUT, MODE>), ClusterSmem<BN>::kAlloc, kClusterThreads};
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

}  // namespace linear
}  // namespace dtg
