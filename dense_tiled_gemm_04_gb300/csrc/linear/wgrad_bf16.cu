// Weight gradients of bf16 operands.
#include "tile_set.cuh"

namespace dtg {
namespace linear {
KernelChoice wgrad_bf16(int config, bool out_f32)
{
    return out_f32 ? tile_choice_for<1, kOutF32, kWgrad, true>(config) : tile_choice_for<1, kOutBf16, kWgrad, false>(config);
}
}  // namespace linear
}  // namespace dtg
