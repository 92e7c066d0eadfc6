// Forward products of E4M3 operands over long contractions.
#include "tile_set.cuh"

namespace dtg {
namespace linear {
KernelChoice forward_long_e4m3(int config, bool out_bf16)
{
    return out_bf16 ? tile_choice_for<2, kOutBf16, kForward, true>(config) : tile_choice_for<2, kOutF16, kForward, true>(config);
}
}  // namespace linear
}  // namespace dtg
