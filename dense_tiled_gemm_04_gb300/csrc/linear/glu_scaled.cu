// Gated forward, 8-bit operands with block scales.
#include "tile_set.cuh"

namespace dtg {
namespace linear {
KernelChoice glu_scaled(int config, bool out_bf16)
{
    return out_bf16 ? glu_choice<2, kOutBf16, true, true>(config) : glu_choice<2, kOutF16, true, true>(config);
}
}  // namespace linear
}  // namespace dtg
