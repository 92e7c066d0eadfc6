// Forward products of 8-bit operands with block scales.
#include "tile_set.cuh"

namespace dtg {
namespace linear {
KernelChoice forward_scaled(int config, bool out_bf16)
{
    return out_bf16 ? scaled_choice<kOutBf16, kForward>(config) : scaled_choice<kOutF16, kForward>(config);
}
}  // namespace linear
}  // namespace dtg
