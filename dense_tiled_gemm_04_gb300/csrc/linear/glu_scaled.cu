// Gated forward, 8-bit operands with block scales.
#include "tile_set.cuh"

namespace dtg {
namespace linear {
KernelChoice glu_scaled(int config, bool out_bf16)
{
    return out_bf16 ? scaled_choice<kOutBf16, kGlu>(config) : scaled_choice<kOutF16, kGlu>(config);
}
}  // namespace linear
}  // namespace dtg
