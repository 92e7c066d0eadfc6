// Weight gradients of fp16 operands in that type over many tokens.
#include "tile_set.cuh"

namespace dtg {
namespace linear {
KernelChoice wgrad_long_f16(int config) { return tile_choice_for<0, kOutF16, kWgrad, true>(config); }
}  // namespace linear
}  // namespace dtg
