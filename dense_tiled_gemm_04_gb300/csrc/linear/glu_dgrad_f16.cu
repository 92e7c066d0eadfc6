// Gated input gradients, fp16 operands.
#include "tile_set.cuh"

namespace dtg {
namespace linear {
KernelChoice glu_dgrad_f16(int config, bool sums)
{
    return sums ? glu_dgrad_choice<0, kOutF16, true>(config) : glu_dgrad_choice<0, kOutF16, false>(config);
}
}  // namespace linear
}  // namespace dtg
