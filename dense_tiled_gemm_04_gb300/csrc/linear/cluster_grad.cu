// Gradients on few tiles.
#include "cluster_set.cuh"

namespace dtg {
namespace linear {
KernelChoice cluster_dgrad(int tokens, bool bf16)
{
    return bf16 ? cluster_choice_for<1, kOutBf16, kDgrad>(tokens) : cluster_choice_for<0, kOutF16, kDgrad>(tokens);
}

KernelChoice cluster_wgrad(bool bf16, bool out_f32)
{
    if (bf16) return out_f32 ? cluster_choice_for<1, kOutF32, kWgrad>(128) : cluster_choice_for<1, kOutBf16, kWgrad>(128);
    return out_f32 ? cluster_choice_for<0, kOutF32, kWgrad>(128) : cluster_choice_for<0, kOutF16, kWgrad>(128);
}
}  // namespace linear
}  // namespace dtg
