// Products on few tiles, 8-bit operands with block scales.
#include "cluster_set.cuh"

namespace dtg {
namespace linear {
KernelChoice cluster_scaled(int tokens, bool out_bf16)
{
    return out_bf16 ? cluster_choice_narrow<2, kOutBf16, kForward, true>(tokens) : cluster_choice_narrow<2, kOutF16, kForward, true>(tokens);
}

KernelChoice cluster_glu_scaled(int tokens, bool out_bf16)
{
    return out_bf16 ? cluster_choice_narrow<2, kOutBf16, kGlu, true>(tokens) : cluster_choice_narrow<2, kOutF16, kGlu, true>(tokens);
}
}  // namespace linear
}  // namespace dtg
