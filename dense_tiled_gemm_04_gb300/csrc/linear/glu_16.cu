// Gated forward, 16-bit operands.
#include "tile_set.cuh"

namespace dtg {
namespace linear {
KernelChoice glu_16(int config, bool bf16, bool sums)
{
    if (bf16) return sums ? glu_choice<1, kOutBf16, true>(config) : glu_choice<1, kOutBf16, false>(config);
    return sums ? glu_choice<0, kOutF16, true>(config) : glu_choice<0, kOutF16, false>(config);
}
}  // namespace linear
}  // namespace dtg
