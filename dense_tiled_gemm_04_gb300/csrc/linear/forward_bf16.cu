// Forward products of bf16 operands.
#include "tile_set.cuh"

namespace dtg {
namespace linear {
KernelChoice forward_bf16(int config) { return tile_choice_for<1, kOutBf16, kForward, false>(config); }
}  // namespace linear
}  // namespace dtg
