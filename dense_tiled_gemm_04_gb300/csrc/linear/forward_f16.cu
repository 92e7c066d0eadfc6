// Forward products of fp16 operands.
#include "tile_set.cuh"

namespace dtg {
namespace linear {
KernelChoice forward_f16(int config) { return tile_choice_for<0, kOutF16, kForward, false>(config); }
}  // namespace linear
}  // namespace dtg
