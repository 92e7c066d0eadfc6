// Forward products of bf16 operands over long contractions.
#include "tile_set.cuh"

namespace dtg {
namespace linear {
KernelChoice forward_long_bf16(int config) { return tile_choice_for<1, kOutBf16, kForward, true>(config); }
}  // namespace linear
}  // namespace dtg
