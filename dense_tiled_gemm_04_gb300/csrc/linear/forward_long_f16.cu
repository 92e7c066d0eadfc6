// Forward products of fp16 operands over long contractions.
#include "tile_set.cuh"

namespace dtg {
namespace linear {
KernelChoice forward_long_f16(int config) { return tile_choice_for<0, kOutF16, kForward, true>(config); }
}  // namespace linear
}  // namespace dtg
