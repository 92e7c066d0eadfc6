// Input gradients through an activation.
#include "tile_set.cuh"

namespace dtg {
namespace linear {
KernelChoice dgrad_16(int config, bool bf16)
{
    return bf16 ? tile_choice_for<1, kOutBf16, kDgrad>(config) : tile_choice_for<0, kOutF16, kDgrad>(config);
}
}  // namespace linear
}  // namespace dtg
