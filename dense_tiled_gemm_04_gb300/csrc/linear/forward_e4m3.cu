// Forward products of E4M3 operands.
#include "tile_set.cuh"

namespace dtg {
namespace linear {
KernelChoice forward_e4m3(int config, bool out_bf16)
{
    return out_bf16 ? tile_choice_for<2, kOutBf16, kForward, false>(config) : tile_choice_for<2, kOutF16, kForward, false>(config);
}
}  // namespace linear
}  // namespace dtg
