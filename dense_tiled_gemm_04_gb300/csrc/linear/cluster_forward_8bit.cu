// Forward products on few tiles, 8-bit operands.
#include "cluster_set.cuh"

namespace dtg {
namespace linear {
KernelChoice cluster_forward_8(int tokens, bool e5m2, bool out_bf16)
{
    if (e5m2)
        return out_bf16 ? cluster_choice_for<3, kOutBf16, kForward>(tokens) : cluster_choice_for<3, kOutF16, kForward>(tokens);
    return out_bf16 ? cluster_choice_for<2, kOutBf16, kForward>(tokens) : cluster_choice_for<2, kOutF16, kForward>(tokens);
}
}  // namespace linear
}  // namespace dtg
