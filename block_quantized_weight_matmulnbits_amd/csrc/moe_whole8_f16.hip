// moe_whole8_f16.hip -- experts' projections of 8-bit codes as whole numbers and f16 inputs.
#include "moe.h"

namespace qmm {

hipError_t launch_moe_whole8_f16(const MoeArgs& a, const MoeWork& w, const MoeSide& side) {
  return launch_moe_scales<DT_F16, 8, true>(a, w, side);
}

}  // namespace qmm
