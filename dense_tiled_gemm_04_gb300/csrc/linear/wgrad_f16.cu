// Weight gradients of fp16 operands.
#include "tile_set.cuh"

namespace dtg {
namespace linear {
KernelChoice wgrad_f16(int config, bool out_f32)
{
    return out_f32 ? tile_choice_for<0, kOutF32, kWgrad, true>(config) : tile_choice_for<0, kOutF16, kWgrad, false>(config);
}
}  // namespace linear
}  // namespace dtg
