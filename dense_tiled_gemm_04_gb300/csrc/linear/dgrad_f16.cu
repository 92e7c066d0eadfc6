// Input gradients through an activation, fp16 operands.
#include "tile_set.cuh"

namespace dtg {
namespace linear {
KernelChoice dgrad_f16(int config, bool sums)
{
    return sums ? tile_choice_for<0, kOutF16, kDgrad, true>(config) : tile_choice_for<0, kOutF16, kDgrad, false>(config);
}
}  // namespace linear
}  // namespace dtg
