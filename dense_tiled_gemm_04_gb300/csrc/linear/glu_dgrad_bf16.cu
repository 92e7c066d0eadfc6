// Gated input gradients, bf16 operands.
#include "tile_set.cuh"

namespace dtg {
namespace linear {
KernelChoice glu_dgrad_bf16(int config, bool sums)
{
    return sums ? glu_dgrad_choice<1, kOutBf16, true>(config) : glu_dgrad_choice<1, kOutBf16, false>(config);
}
}  // namespace linear
}  // namespace dtg
