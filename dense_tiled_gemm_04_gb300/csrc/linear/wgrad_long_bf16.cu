// Weight gradients of bf16 operands in that type over many tokens.
#include "tile_set.cuh"

namespace dtg {
namespace linear {
KernelChoice wgrad_long_bf16(int config) { return tile_choice_for<1, kOutBf16, kWgrad, true>(config); }
}  // namespace linear
}  // namespace dtg
