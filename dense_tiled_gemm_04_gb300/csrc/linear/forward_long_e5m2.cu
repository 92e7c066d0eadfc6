// Forward products of E5M2 operands over long contractions.
#include "tile_set.cuh"

namespace dtg {
namespace linear {
KernelChoice forward_long_e5m2(int config, bool out_bf16)
{
    return out_bf16 ? tile_choice_for<3, kOutBf16, kForward, true>(config) : tile_choice_for<3, kOutF16, kForward, true>(config);
}
}  // namespace linear
}  // namespace dtg
