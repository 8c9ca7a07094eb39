// moe_whole8_bf16.hip -- experts' projections of 8-bit codes as whole numbers and bf16 inputs.
#include "moe.h"

namespace qmm {

hipError_t launch_moe_whole8_bf16(const MoeArgs& a, const MoeWork& w, const MoeSide& side) {
  return launch_moe_scales<DT_BF16, 8, true>(a, w, side);
}

}  // namespace qmm
