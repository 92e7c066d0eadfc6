// Gated products on few tiles, 16-bit operands.
#include "cluster_set.cuh"

namespace dtg {
namespace linear {
KernelChoice cluster_glu_16(int tokens, bool bf16)
{
    return bf16 ? cluster_choice_narrow<1, kOutBf16, kGlu, false>(tokens) : cluster_choice_narrow<0, kOutF16, kGlu, false>(tokens);
}

KernelChoice cluster_glu_dgrad(bool bf16)
{
    return bf16 ? cluster_choice<64, 1, kOutBf16, kGluDgrad>() : cluster_choice<64, 0, kOutF16, kGluDgrad>();
}
}  // namespace linear
}  // namespace dtg
