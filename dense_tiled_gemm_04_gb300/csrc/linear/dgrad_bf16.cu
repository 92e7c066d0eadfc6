// Input gradients through an activation, bf16 operands.
#include "tile_set.cuh"

namespace dtg {
namespace linear {
KernelChoice dgrad_bf16(int config, bool sums)
{
    return sums ? tile_choice_for<1, kOutBf16, kDgrad, true>(config) : tile_choice_for<1, kOutBf16, kDgrad, false>(config);
}
}  // namespace linear
}  // namespace dtg
