// Forward products on few tiles, 16-bit operands.
#include "cluster_set.cuh"

namespace dtg {
namespace linear {
KernelChoice cluster_forward_16(int tokens, bool bf16)
{
    return bf16 ? cluster_choice_for<1, kOutBf16, kForward>(tokens) : cluster_choice_for<0, kOutF16, kForward>(tokens);
}
}  // namespace linear
}  // namespace dtg
